"""The paged operators on the GPU against plain 64-bit implementations
(paged_reference): rotation and append with several axes, attention with capped
scores, bias and masks, shared prefixes; and all of them run together."""
import numpy as np
import pytest

import oracle
import workloads as W
import chunked_prefill_mixed_gb300 as S
import paged_reference as R

pytestmark = pytest.mark.gpu

HEADS = [(4, 4, 64), (8, 2, 64), (8, 4, 128), (10, 2, 128), (7, 1, 64), (14, 2, 128), (16, 1, 128), (6, 3, 128)]


def _runner(Hq, Hkv, d, dtype, **kw):
    from chunked_prefill_mixed_gb300.runner import PagedRunner
    return PagedRunner(Hq, Hkv, d, dtype=R.torch_type(dtype), **kw)


def _values(rng, dtype, *shape, scale=1.0):
    import torch
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to("cuda").to(R.torch_type(dtype))


class Attn:
    """A batch's tensors on the GPU, one call, and the check against 64 bits."""

    def __init__(self, b, Hq, Hkv, d, dtype, seed=0, cap=0.0, slopes=False, sms=None, qscale=1.5):
        import torch
        rng = np.random.default_rng(seed)
        self.b, self.dtype, self.d, self.cap = b, dtype, d, cap
        self.T = int(b["qo"][-1])
        self.q = _values(rng, dtype, self.T, Hq, d, scale=qscale)
        self.kc, self.vc = (_values(rng, dtype, b["pages"], Hkv, 16, d) for _ in range(2))
        self.k64, self.v64 = R.to64(self.kc), R.to64(self.vc)
        self.spoil()
        self.slopes = None
        if slopes:
            self.slopes = torch.from_numpy((2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)).cuda()
        self.r = _runner(Hq, Hkv, d, dtype)
        if sms:
            self.r.num_sms = sms
        args, more = R.plan_args(b)
        self.plan = self.r.plan(*args, **more)
        self.out = torch.full((self.T + 2, Hq, d), 7.0, dtype=self.q.dtype, device="cuda")
        self.lse = torch.full((self.T + 2, Hq), 7.0, dtype=torch.float32, device="cuda")

    def spoil(self):
        """Pages of no row, and the slots past a row's last key, hold NaN."""
        used = set()
        for s, length in enumerate(self.b["len"]):
            ids = self.b["ids"][self.b["ptr"][s]:self.b["ptr"][s + 1]]
            used.update(ids.tolist())
            if length % 16:
                for c in (self.kc, self.vc):
                    c[int(ids[-1]), :, length % 16:] = float("nan")
        for p in set(range(self.b["pages"])) - used:
            self.kc[p] = self.vc[p] = float("nan")

    def call(self, **kw):
        self.r.attend(self.plan, self.q, self.kc, self.vc, self.out, score_cap=self.cap, slopes=self.slopes,
                      lse=self.lse, **kw)

    def check(self, what=""):
        slopes = None if self.slopes is None else self.slopes.cpu().numpy().astype(np.float64)
        ref = R.attention(self.b, R.to64(self.q), self.k64, self.v64, 1 / np.sqrt(self.d), self.cap, slopes)
        R.assert_attention(R.to64(self.out[:self.T]), ref, self.dtype, R.to64(self.lse[:self.T]), what)
        assert bool((self.out[self.T:] == 7.0).all()) and bool((self.lse[self.T:] == 7.0).all()), "rows past the batch"
        return ref

    def run(self, what=""):
        self.call()
        assert self.r.status() == 0
        return self.check(what)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_ragged_causal(heads, dtype):
    rng = np.random.default_rng(1)
    b = R.make_batch(rng, [1, 5, 1, 37, 1, 130, 16, 1], [1, 5, 17, 100, 300, 130, 144, 128])
    Attn(b, *heads, dtype).run()


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("new", [1, 2, 9, 128, 1000])
def test_lengths(new, length):
    rng = np.random.default_rng(length)
    b = R.make_batch(rng, [min(new, length)], [length])
    Attn(b, 8, 2, 128 if length % 2 else 64, "bf16" if new % 2 else "fp16").run(f"{new} of {length}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap,slopes", [(0.0, True), (2.0, False), (30.0, False), (50.0, True)])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 4, 128), (14, 2, 128)], ids=str)
def test_cap_and_bias(heads, cap, slopes, dtype):
    rng = np.random.default_rng(2)
    b = R.make_batch(rng, [1, 70, 1, 260, 3], [90, 333, 700, 260, 515], prefix_len=[0, 0, 0, 100, 0])
    Attn(b, *heads, dtype, cap=cap, slopes=slopes, qscale=6.0 if cap else 1.5).run()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap", [0.01, 0.5, 100.0, 200.0, 1000.0, 1e5, 1e9])
def test_caps_far_from_the_scores(cap, dtype):
    """From caps that saturate every score to caps that leave the scores as they are."""
    rng = np.random.default_rng(21)
    b = R.make_batch(rng, [1, 70, 1, 3], [90, 333, 700, 515])
    for d, qscale in ((64, 2.0), (128, 12.0)):
        Attn(b, 8, 2, d, dtype, cap=cap, qscale=qscale).run(f"d {d}, scores times {qscale}")


@pytest.mark.parametrize("cap,scale", [(0.0, 1e-3), (0.0, 3.0), (20.0, 1e-3), (20.0, 4.0), (300.0, 4.0), (0.05, 4.0)])
def test_scales(cap, scale):
    rng = np.random.default_rng(22)
    b = R.make_batch(rng, [1, 70, 1, 3], [90, 333, 700, 515])
    x = Attn(b, 8, 4, 128, "fp16", cap=cap, qscale=0.3)
    x.call(sm_scale=scale)
    assert x.r.status() == 0
    ref = R.attention(b, R.to64(x.q), x.k64, x.v64, scale, cap)
    R.assert_attention(R.to64(x.out[:x.T]), ref, "fp16", R.to64(x.lse[:x.T]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights(first, new, dtype):
    """One key outweighs each of the 60000 others 10^7 times, and has the value 0:
    the output is the others' share, each weight below fp16's normal numbers."""
    import torch
    d, length = 64, 60000
    b = R.make_batch(np.random.default_rng(23), [new], [length], key_lo=np.zeros(new, np.int32),
                     key_hi=np.full(new, length, np.int32), permute=False)
    x = Attn(b, 4, 4, d, dtype)
    x.q.zero_(), x.kc.zero_(), x.vc.zero_()
    x.q[..., 0] = 16.0
    x.vc[:, :, :] = 1.0
    at = 0 if first else length - 1
    page = int(b["ids"][at // 16])
    x.kc[page, :, at % 16, 0] = 8.0625       # a score of 16.125 beside 0
    x.vc[page, :, at % 16] = 0.0
    x.call()
    assert x.r.status() == 0
    share = (length - 1) / (length - 1 + np.exp(16.125))
    # weight and output rounding; twice 2^-18 for the exponentials, 2^-22 each of the
    # logits of 23.3, and for the sum
    tol = share * (2.2 * R.U[dtype] + 2.0 ** -17)
    assert abs(R.to64(x.out[:x.T]) - share).max() <= tol


def test_rows_done_again_over_long_contexts():
    """The last token's value is infinite: the others of its tile do not see it, and
    have a long context of their own."""
    rng = np.random.default_rng(24)
    b = R.make_batch(rng, [40], [9000])
    for d, dtype in ((64, "bf16"), (128, "fp16")):
        x = Attn(b, 4, 2, d, dtype, cap=30.0)
        page = int(b["ids"][-1])
        x.vc[page, :, (9000 - 1) % 16] = float("inf")
        x.call()
        assert x.r.status() == 0
        ref = R.attention(b, R.to64(x.q), x.k64, x.v64, 1 / np.sqrt(d), 30.0)
        R.assert_attention(R.to64(x.out[:39]), [y[:39] for y in ref], dtype, R.to64(x.lse[:39]))
        assert bool((x.out[39] == float("inf")).all())


@pytest.mark.parametrize("window", [1, 2, 16, 100, 300, 5000])
def test_window(window):
    rng = np.random.default_rng(3)
    b = R.make_batch(rng, [1, 70, 1, 260, 1], [90, 333, 700, 260, 515], window=window)
    Attn(b, 8, 4, 128, "bf16").run()


@pytest.mark.parametrize("prefix", [1, 60, 128, 259, 400])
def test_prefix(prefix):
    rng = np.random.default_rng(4)
    b = R.make_batch(rng, [1, 70, 260, 40], [90, 333, 260, 40], prefix_len=[prefix] * 4, window=0)
    Attn(b, 8, 2, 128, "fp16").run()
    b["window"] = 33
    Attn(b, 8, 2, 64, "bf16", slopes=True).run()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_documents_and_rows_that_see_nothing(dtype):
    rng = np.random.default_rng(5)
    n, length = [300, 1, 64, 1, 20], [420, 33, 64, 200, 20]
    b = R.make_batch(rng, n, length)
    lo, hi = [], []
    for k, (a, z) in enumerate(zip(n, length)):
        for p in range(z - a, z):
            lo.append(p // 50 * 50)
            hi.append(p + 1)
    lo, hi = np.array(lo, np.int32), np.array(hi, np.int32)
    lo[10:40] = hi[10:40]              # empty, in a tile with others
    lo[40:50], hi[40:50] = 300, 20     # lo past hi
    hi[60:64], lo[64:66] = -5, 10 ** 6  # outside the row
    lo[300] = 33                        # an empty one-token row
    hi[301:365] = 0                     # a whole row of 64 tokens empty
    hi[366:386] = 20                    # every token sees every key
    b.update(key_lo=lo, key_hi=hi)
    for heads in ((8, 2, 64), (14, 2, 128)):
        Attn(b, *heads, dtype).run()


def test_unseen_keys_may_hold_anything():
    """Infinities, NaN and the largest values in keys and values that a token does
    not see: later tokens of its own chunk, other documents, before its window."""
    import torch
    rng = np.random.default_rng(6)
    for dtype in ("bf16", "fp16"):
        n, length = [200, 150, 1, 40], [200, 300, 64, 170]
        lo = np.concatenate([np.arange(z - a, z) // 32 * 32 for a, z in zip(n, length)]).astype(np.int32)
        b = R.make_batch(rng, n, length, key_lo=lo)
        x = Attn(b, 8, 2, 128, dtype)
        big = torch.finfo(x.q.dtype).max
        for s in range(4):
            ids = b["ids"][b["ptr"][s]:b["ptr"][s + 1]]
            for j, val in ((5, float("nan")), (33, float("inf")), (40, -float("inf")), (63, big), (100, float("nan"))):
                if j < length[s]:
                    for c in (x.kc, x.vc):
                        c[int(ids[j // 16]), :, j % 16] = val
        x.call()
        assert x.r.status() == 0
        # tokens that see a spoilt key are left out of the comparison
        bad = np.zeros(x.T, bool)
        for t, (s, p, a, z) in enumerate(R.intervals(b)):
            bad[t] = any(a <= j < z and j < length[s] for j in (5, 33, 40, 63, 100))
        assert 20 < (~bad).sum() < x.T
        ref = R.attention(b, R.to64(x.q), x.k64, x.v64, 1 / np.sqrt(128))
        keep = ~bad
        R.assert_attention(R.to64(x.out[:x.T])[keep], tuple(r[keep] for r in ref), dtype,
                           R.to64(x.lse[:x.T])[keep], dtype)


@pytest.mark.parametrize("sms", [1, 7, 1000])
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64), (3, 3, 128)], ids=str)
def test_work_split_along_the_keys(heads, sms):
    """A plan for many SMs cuts the keys into pieces, one for few does not: the
    same results, and the same bits from call to call."""
    import torch
    rng = np.random.default_rng(7)
    b = R.make_batch(rng, [1, 1, 200, 1, 3], [5000, 40, 2100, 1029, 900], window=4000)
    x = Attn(b, *heads, "bf16", sms=sms, slopes=True)
    x.run()
    first, lse = x.out.clone(), x.lse.clone()
    for _ in range(3):
        x.out.fill_(7.0)
        x.call()
        torch.cuda.synchronize()
        assert torch.equal(x.out, first) and torch.equal(x.lse, lse)


def test_strided_queries_and_contiguous_pages():
    rng = np.random.default_rng(8)
    b = R.make_batch(rng, [1, 300, 1, 17], [900, 640, 31, 1700], permute=False)
    x = Attn(b, 8, 2, 128, "bf16")
    whole = _values(rng, "bf16", x.T, 12, 128)
    x.q = whole[:, 2:10]
    x.run()


# ------------------------------------------------------------------ shared prefixes
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (14, 2, 128), (16, 1, 64)], ids=str)
@pytest.mark.parametrize("sms", [4, 152, 900])
def test_shared_prefix(heads, dtype, sms):
    rng = np.random.default_rng(9)
    length = [40 * 16 + 3, 40 * 16 + 16, 40 * 16 + 200, 60, 9 * 16 + 1, 9 * 16 + 90, 5, 700]
    n = [1, 1, 1, 1, 1, 60, 2, 1]
    b = R.make_batch(rng, n, length, shared=[((0, 1, 2), 40), ((4, 5), 9)],
                     group_indptr=np.array([0, 3, 4, 6], np.int32), group_pages=np.array([40, 0, 9], np.int32))
    x = Attn(b, *heads, dtype, sms=sms, cap=20.0, slopes=True)
    x.run()
    plain = {k: v for k, v in b.items() if not k.startswith("group")}
    y = Attn(plain, *heads, dtype, sms=sms, cap=20.0, slopes=True)
    y.run()


@pytest.mark.parametrize("sms", [2, 152])   # (with 152 the small groups are left to their rows)
def test_shared_prefix_with_masks_and_many_rows(sms):
    rng = np.random.default_rng(10)
    rows = 90
    length = [33 * 16 + 1 + int(rng.integers(0, 60)) for _ in range(rows)]
    lo = np.array([int(rng.integers(0, z)) for z in length], np.int32)
    lo[:5] = 33 * 16           # see nothing of the prefix
    lo[5] = length[5]          # see nothing at all
    b = R.make_batch(rng, [1] * rows, length, shared=[(range(rows), 33)], key_lo=lo, share_pages=2)
    x = Attn(b, 8, 2, 128, "bf16", sms=sms)
    assert x.plan.info.n_merge == rows
    x.run()
    # the rows' tails wholly within the shared pages: a group over all their keys
    b = R.make_batch(rng, [1, 1, 1], [64, 64, 64], shared=[(range(3), 4)],
                     group_indptr=np.array([0, 3], np.int32), group_pages=np.array([4], np.int32))
    x = Attn(b, 16, 8, 64, "fp16", sms=sms)
    assert (x.plan.info.n_first > 0) == (sms == 2)
    x.run()


# ------------------------------------------------------------------ append
def _append_case(dtype, Hq, Hkv, d, T, sections, style, seed, max_pos=5000, theta=10000.0, fused=False):
    import torch
    rng = np.random.default_rng(seed)
    if fused:
        whole = _values(rng, dtype, T, Hq + 2 * Hkv, d)
        q, k, v = whole[:, :Hq], whole[:, Hq:Hq + Hkv], whole[:, Hq + Hkv:]
    else:
        q, k, v = (_values(rng, dtype, T, h, d) for h in (Hq, Hkv, Hkv))
    pages = T // 16 + 3
    kc, vc = (_values(rng, dtype, pages, Hkv, 16, d) for _ in range(2))
    slots = rng.permutation(pages * 16)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    pos = rng.integers(0, max_pos, size=(len(sections), T)).astype(np.int32)
    pos[:, :1] = max_pos - 1
    r = _runner(Hq, Hkv, d, dtype, max_pos=max_pos, rope_theta=theta, rope_style=style)
    q_out = torch.full((T, Hq, d), 7.0, dtype=q.dtype, device="cuda")
    k0, v0 = R.to64(kc), R.to64(vc)
    r.append(k, v, kc, vc, torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), q=q, q_out=q_out,
             sections=sections)
    assert r.status() == 0
    ang = R.angles(pos, sections, d, theta)
    live = slots >= 0
    k0[slots[live] // 16, :, slots[live] % 16] = R.round_to(R.rotate(R.to64(k), ang, style), dtype)[live]
    v0[slots[live] // 16, :, slots[live] % 16] = R.to64(v)[live]
    assert np.array_equal(R.to64(vc), v0), "values"
    assert np.array_equal(R.to64(kc), k0), f"{(R.to64(kc) != k0).sum()} key elements differ"
    want = R.rotate(R.to64(q), ang, style)
    got = R.to64(q_out)
    assert np.all(got[~live] == 7.0), "a skipped token's query was written"
    # rotated in fp32 (three roundings and the table's, of the pair's magnitude), rounded once
    half = d // 2
    x = np.abs(R.to64(q))
    mag = x + (np.concatenate([x[..., half:], x[..., :half]], -1) if style == 0
               else x.reshape(T, Hq, half, 2)[..., ::-1].reshape(x.shape))
    tol = R.U[dtype] * np.abs(want) + 1.01 * 2.0 ** -22 * mag + (2.0 ** -25 if dtype == "fp16" else 0)
    assert np.all(np.abs(got - want)[live] <= tol[live])


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (14, 2, 128), (16, 1, 64)], ids=str)
def test_append_bits(heads, dtype, style):
    Hq, Hkv, d = heads
    _append_case(dtype, Hq, Hkv, d, 700, [d // 2], style, 1)
    a = d // 8
    _append_case(dtype, Hq, Hkv, d, 300, [a, 3, d // 2 - a - 3], style, 2, fused=True)


@pytest.mark.parametrize("tokens", [1, 2, 3, 37, 39, 1000, 5000])
def test_append_token_counts(tokens):
    _append_case("bf16", 32, 8, 128, tokens, [64], 0, tokens, max_pos=131072, theta=500000.0)
    _append_case("fp16", 8, 1, 64, tokens, [8, 8, 8, 8], 0, tokens)


def test_append_small_and_large_values():
    """Elements where the rounding to the type is at its edges: subnormals of fp16,
    zeros, values near the type's largest."""
    import torch
    rng = np.random.default_rng(3)
    for dtype in ("bf16", "fp16"):
        T, Hkv, d = 400, 2, 64
        k = rng.standard_normal((T, Hkv, d)) * 10.0 ** rng.integers(-9 if dtype == "fp16" else -41, 4, size=(T, 1, 1))
        k[5], k[6, :, ::2], k[7] = 0.0, 0.0, 30000.0
        kt = torch.from_numpy(k.astype(np.float32)).cuda().to(R.torch_type(dtype))
        kc, vc = torch.zeros(30, Hkv, 16, d, dtype=kt.dtype, device="cuda"), torch.zeros(30, Hkv, 16, d, dtype=kt.dtype, device="cuda")
        slots, pos = np.arange(T, dtype=np.int32), rng.integers(0, 3000, (1, T)).astype(np.int32)
        r = _runner(4, Hkv, d, dtype, max_pos=3000)
        r.append(kt, kt, kc, vc, torch.from_numpy(slots).cuda(), torch.from_numpy(pos[0].copy()).cuda())
        assert r.status() == 0
        want = R.round_to(R.rotate(R.to64(kt), R.angles(pos, [d // 2], d, 10000.0)), dtype)
        got = R.to64(kc).transpose(0, 2, 1, 3).reshape(-1, Hkv, d)[:T]
        assert np.array_equal(got, want)


def test_append_queries_in_place_and_without():
    import torch
    rng = np.random.default_rng(4)
    T, Hq, Hkv, d = 50, 8, 2, 128
    q, k, v = (_values(rng, "bf16", T, h, d) for h in (Hq, Hkv, Hkv))
    r = _runner(Hq, Hkv, d, "bf16", max_pos=100)
    slots, pos = (torch.arange(T, dtype=torch.int32, device="cuda") for _ in range(2))
    pools = [torch.zeros(4, Hkv, 16, d, dtype=q.dtype, device="cuda") for _ in range(4)]
    out = torch.empty_like(q)
    r.append(k, v, pools[0], pools[1], slots, pos, q=q, q_out=out)
    r.append(k, v, pools[2], pools[3], slots, pos, q=q, q_out=q)
    assert torch.equal(out, q)
    r.append(k, v, pools[2].zero_(), pools[3].zero_(), slots, pos)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    r.append(k[:0], v[:0], pools[2], pools[3], slots[:0], pos[:0])
    assert r.status() == 0


# ------------------------------------------------------------------ device-side checks
def test_bad_pages_slots_and_positions_are_reported():
    import torch
    rng = np.random.default_rng(11)
    # append: a slot past the pool, a position past the table, a negative one
    T, Hq, Hkv, d = 20, 4, 2, 64
    k = _values(rng, "bf16", T, Hkv, d)
    r = _runner(Hq, Hkv, d, "bf16", max_pos=64)
    for slot, p in ((3 * 16, 5), (5, 64), (5, -1), (2 ** 31 - 1, 5)):
        kc, vc = (torch.zeros(3, Hkv, 16, d, dtype=k.dtype, device="cuda") for _ in range(2))
        slots, pos = (torch.arange(T, dtype=torch.int32, device="cuda") for _ in range(2))
        slots[7], pos[7] = slot, p
        r.append(k, k, kc, vc, slots, pos)
        assert r.status() == 2 and r.status() == 0
        flat = vc.transpose(1, 2).reshape(-1, Hkv, d)
        keep = [i for i in range(T) if i != 7]
        assert torch.equal(flat[keep], k[keep]) and not bool(flat[7].any())
    # attention: page ids outside the pool, in a decode, a chunk and a shared prefix
    for row, more in ((0, {}), (1, {}), (0, dict(share_pages=3))):
        b = R.make_batch(rng, [1, 150, 1], [300, 400, 250], shared=[((0, 2), 10)] if more else None)
        if more:
            b = R.make_batch(rng, [1, 1, 1], [300, 260, 250], shared=[((0, 1, 2), 10)], **more)
        for bad in (b["pages"], -1):
            x = Attn(b, 8, 2, 128, "bf16", sms=4 if more else None)
            good = x.plan.dev.clone()
            at = x.plan.info.off_pages + int(b["ptr"][row]) + 1
            x.plan.dev[at] = bad
            x.call()
            assert x.r.status() == 2
            x.plan.dev.copy_(good)
            x.run("after an error")


# ------------------------------------------------------------------ streams and graphs
def test_streams_and_graphs():
    import torch
    rng = np.random.default_rng(12)
    b = R.make_batch(rng, [1, 1, 100, 1], [3000, 40, 600, 777])
    x = Attn(b, 8, 2, 128, "bf16", sms=600)
    x.run()
    want = x.out.clone()
    # two streams at once
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(x.out) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip((s1, s2), outs):
            x.r.attend(x.plan, x.q, x.kc, x.vc, o, stream=s)
    torch.cuda.synchronize()
    assert x.r.status() == 0
    for o in outs:
        assert torch.equal(o[:x.T], want[:x.T])
    # two graphs of one runner, replayed one after the other, with changed inputs
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.r.attend(x.plan, x.q, x.kc, x.vc, o)
        graphs.append(g)
    for trial in range(3):
        for o in outs:
            o.zero_()
        if trial:
            x.q.copy_(_values(rng, "bf16", *x.q.shape, scale=1.5))
        for g in graphs:
            g.replay()
        x.call()
        torch.cuda.synchronize()
        assert x.r.status() == 0
        for o in outs:
            assert torch.equal(o[:x.T], x.out[:x.T])
    x.check()


def test_threads_share_a_runner():
    """Calls of two threads on one stream, each a kernel and the join of its partial rows."""
    import threading
    rng = np.random.default_rng(14)
    xs = [Attn(R.make_batch(rng, [1, 1], [4000, n]), 8, 2, 128, "bf16", seed=n, sms=600) for n in (3500, 2900)]
    r = xs[0].r
    plans = []
    for x in xs:
        args, more = R.plan_args(x.b)
        plans.append(r.plan(*args, **more))
        assert plans[-1].info.n_merge == 2
        x.run()
    wants = [x.out.clone() for x in xs]
    failed = []

    def work(x, plan, want):
        for _ in range(50):
            x.out.fill_(7.0)
            r.attend(plan, x.q, x.kc, x.vc, x.out)
            if not bool((x.out == want).all()):
                failed.append(1)
    threads = [threading.Thread(target=work, args=a) for a in zip(xs, plans, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and r.status() == 0


def test_plan_used_and_dropped_on_another_stream():
    import torch
    rng = np.random.default_rng(15)
    b = R.make_batch(rng, [1, 30], [400, 100])
    x = Attn(b, 8, 2, 128, "bf16")
    x.run()
    want, side = x.out.clone(), torch.cuda.Stream()
    x.out.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    x.call(stream=side)
    n = x.plan.dev.numel()
    del x.plan
    new = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(4)]  # (where the plan was, if it were free)
    torch.cuda.synchronize()
    assert x.r.status() == 0 and torch.equal(x.out, want) and len(new) == 4


def test_capture_on_a_stream_that_joins_the_current_one():
    import torch
    rng = np.random.default_rng(16)
    x = Attn(R.make_batch(rng, [1, 30], [4000, 100]), 8, 2, 128, "bf16", sms=400)
    x.run()
    want, side = x.out.clone(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        x.call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    assert not x.r._others
    for _ in range(3):
        x.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.out, want)
    assert x.r.status() == 0


def test_calls_that_follow_one_another_see_what_is_before_them():
    """Launches overlap the end of the kernel before them: back to back, eager and
    captured, each must still see the inputs that a copy, an append or another
    attention wrote right before it."""
    import torch
    rng = np.random.default_rng(13)
    b = R.make_batch(rng, [1, 1, 1, 40], [2500, 900, 17, 300], shared=[((0, 1), 50)], share_pages=4)
    x = Attn(b, 8, 2, 128, "bf16", sms=400)
    r, T = x.r, x.T
    r.rope = torch.empty(2 * 64 * 128, dtype=torch.float64, device="cuda")
    S.sarathi_rope_table(r.rope, 64, 128, 10000.0, torch.cuda.current_stream())
    r.max_pos, r._append = 64, S.append_args(r.rope, 64, r.shape)
    xs = [_values(rng, "bf16", T, 8, 128) for _ in range(3)]
    k = _values(rng, "bf16", T, 2, 128)
    scratch = [torch.zeros(8, 2, 16, 128, dtype=k.dtype, device="cuda") for _ in range(2)]
    slots, pos = (torch.arange(T, dtype=torch.int32, device="cuda") for _ in range(2))
    q, mid = torch.empty_like(xs[0]), torch.empty_like(xs[0])
    outs = [torch.empty_like(q) for _ in range(3)]

    def chain():
        for src, out in zip(xs, outs):
            q.copy_(src)                                                    # a copy
            r.append(k, k, *scratch, slots, pos, q=q, q_out=q)              # rotates q in place
            r.attend(x.plan, q, x.kc, x.vc, mid)
            r.attend(x.plan, mid, x.kc, x.vc, out)                          # reads the one before
    want = []
    for src in xs:
        q.copy_(src)
        torch.cuda.synchronize()
        r.append(k, k, *scratch, slots, pos, q=q, q_out=q)
        torch.cuda.synchronize()
        r.attend(x.plan, q, x.kc, x.vc, mid)
        torch.cuda.synchronize()
        out = torch.empty_like(q)
        r.attend(x.plan, mid, x.kc, x.vc, out)
        torch.cuda.synchronize()
        want.append(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for call in (chain, g.replay) * 4:
        for o in outs:
            o.zero_()
        call()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert r.status() == 0


# ------------------------------------------------------------------ together, as they are used
def _step_batch(wl):
    st, meta = oracle.plan(*wl.arrays(), wl.budget, 16)
    return meta


@pytest.mark.parametrize("shape", [W.Shape(8, 2, 64), W.Shape(16, 4, 128)], ids=str)
def test_append_then_attend_gives_the_mixed_step(shape):
    """A plan's step by the fused kernel, and by slot mapping, append and paged
    attention: the same page bits, outputs within the step's tolerance."""
    import torch
    from gpu_helpers import GpuStep, assert_close, to_u16
    specs = [(W.DECODE, 0, 40, 41), (W.DECODE, 0, 1070, 1071), (W.PREFILL_RUNNING, 500, 64, 500),
             (W.PREFILL_WAITING, 170, 0, 170)]
    gs = GpuStep(W._build("paged_step", shape, 400, specs, 21, permute=True, spare_pages=2))
    kc, vc = gs.kc_dev.clone(), gs.vc_dev.clone()
    assert gs.run() == 0
    r = _runner(shape.H_q, shape.H_kv, shape.d, "bf16", max_pos=gs.runner.max_pos)
    slots, pos = S.sarathi_slot_mapping(gs.info, gs.packed)
    q = torch.empty_like(gs.q_dev)
    r.append(gs.k_dev, gs.v_dev, kc, vc, torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), q=gs.q_dev,
             q_out=q)
    m = S.plan_arrays(gs.info, gs.packed)
    plan = r.plan(m["qo_indptr"], m["kv_page_indptr"], m["kv_page_indices"], m["kv_last_page_len"])
    out = torch.empty_like(gs.out)
    r.attend(plan, q, kc, vc, out)
    assert r.status() == 0
    assert torch.equal(kc, gs.kc_dev) and torch.equal(vc, gs.vc_dev)
    ref, rt, rh = gs.oracle_rows(*gs.oracle_caches())
    assert_close(oracle.bf16_to_double(to_u16(out))[rt, rh], ref, "append + attend")


def test_project_append_attend_over_steps_with_a_shared_prompt():
    """A shared system prompt is prefilled in chunks, then three requests decode
    behind it: projection, append (three-axis positions), attention with the
    prompt's pages shared, checked at every step in 64 bits."""
    import torch
    rng = np.random.default_rng(31)
    Hq, Hkv, d, hidden, sections = 8, 2, 128, 256, (16, 24, 24)
    shape = S.Shape(Hq, Hkv, d, 16)
    r = _runner(Hq, Hkv, d, "bf16", max_pos=512)
    w = _values(rng, "bf16", (Hq + 2 * Hkv) * d, hidden, scale=hidden ** -0.5)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kc, vc = (torch.full((40, Hkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    prompt, tables = 80, [list(range(5)) + [10 + 8 * i + j for j in range(8)] for i in range(3)]

    def step(rows, share):
        """rows: (request, history, new tokens)."""
        T = sum(n for _, _, n in rows)
        x = _values(rng, "bf16", T, hidden)
        q, k, v = (torch.empty(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
        S.sarathi_qkv_proj(x, w, q, k, v, shape, ws, torch.cuda.current_stream())
        at = [(i, h + a) for i, h, n in rows for a in range(n)]
        slots = np.array([tables[i][p // 16] * 16 + p % 16 for i, p in at], np.int32)
        pos = np.array([[p // 3 for _, p in at], [p % 3 for _, p in at], [p for _, p in at]], np.int32)
        raw = R.to64(q)
        r.append(k, v, kc, vc, torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), q=q, q_out=q,
                 sections=sections)
        length = [h + n for _, h, n in rows]
        per = [-(-z // 16) for z in length]
        b = dict(n=[n for _, _, n in rows], len=length, ptr=np.concatenate([[0], np.cumsum(per)]).astype(np.int32),
                 ids=np.concatenate([tables[i][:c] for (i, _, _), c in zip(rows, per)]).astype(np.int32),
                 qo=np.concatenate([[0], np.cumsum([n for _, _, n in rows])]).astype(np.int32),
                 last=np.array([(z - 1) % 16 + 1 for z in length], np.int32), pages=40)
        plan = r.plan(b["qo"], b["ptr"], b["ids"], b["last"], share_pages=share)
        out = torch.empty_like(q)
        r.attend(plan, q, kc, vc, out, score_cap=30.0)
        assert r.status() == 0
        want_q = R.rotate(raw, R.angles(pos, sections, d, 10000.0))
        assert np.all(np.abs(R.to64(q) - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -20 * (1 + np.abs(raw).max()))
        k64, v64 = np.nan_to_num(R.to64(kc)), np.nan_to_num(R.to64(vc))
        R.assert_attention(R.to64(out), R.attention(b, R.to64(q), k64, v64, d ** -0.5, 30.0), "bf16")
        return plan

    step([(0, 0, 33)], 0)
    step([(0, 33, prompt - 33)], 0)
    for k in range(20):
        plan = step([(i, prompt + k, 1) for i in range(3)], 2)
        assert plan.info.n_merge == 3


@pytest.mark.parametrize("permute", [True, False])
def test_pools_past_two_to_the_31_elements(permute):
    """Appended to and read from pages whose elements' offsets need 64 bits."""
    import torch
    rng = np.random.default_rng(31)
    Hq, Hkv, d, pages = 16, 8, 128, 150_000       # 2.46 10^9 elements a pool
    n, length = [1, 40, 1], [40, 200, 17]
    b = R.make_batch(rng, n, length, permute=permute)
    b["ids"] = (b["ids"] + (pages - b["pages"])).astype(np.int32)
    b["pages"] = pages
    r = _runner(Hq, Hkv, d, "bf16", max_pos=256)
    pools = [torch.empty(pages, Hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    first = int(b["ids"].min())
    for p in pools:
        p[first:] = _values(rng, "bf16", pages - first, Hkv, 16, d)
    T = sum(n)
    k, v = _values(rng, "bf16", T, Hkv, d), _values(rng, "bf16", T, Hkv, d)
    q = _values(rng, "bf16", T, Hq, d)
    at = [(s, z - a + i) for s, (a, z) in enumerate(zip(n, length)) for i in range(a)]
    slots = np.array([int(b["ids"][b["ptr"][s] + p // 16]) * 16 + p % 16 for s, p in at], np.int32)
    pos = np.array([p for _, p in at], np.int32)
    out = torch.empty_like(q)
    r.append(k, v, *pools, torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), q=q, q_out=q)
    args, _ = R.plan_args(b)
    r.attend(r.plan(*args), q, *pools, out)
    assert r.status() == 0
    small = dict(b, ids=b["ids"] - first, pages=pages - first)
    k64, v64 = (R.to64(p[first:]) for p in pools)
    for t, (s, p) in enumerate(at):
        page = int(small["ids"][b["ptr"][s] + p // 16])
        assert np.array_equal(v64[page, :, p % 16], R.to64(v[t]))
    R.assert_attention(R.to64(out), R.attention(small, R.to64(q), k64, v64, 1 / np.sqrt(d)), "bf16")


# ------------------------------------------------------------------ what a token does not see
def _spoilt_values(x, s, key, value):
    """The value row of a key of row s, all kv heads."""
    page = int(x.b["ids"][x.b["ptr"][s] + key // 16])
    x.vc[page, :, key % 16] = value


def _empty_parts(x):
    """(tokens of a tile item that see none of its keys, such items with partial rows,
    such items without)."""
    info, packed = x.plan.info, x.plan.dev.cpu().numpy()
    items = packed[info.off_items:][:info.n_items * 8].reshape(-1, 8)
    toks = packed[info.off_tokens:][:x.T * 4].reshape(-1, 4)
    count, cut, whole = 0, 0, 0
    for kind, _, t0, nt, _, kb, ke, part in items:
        if kind == 0 and kb < ke:
            t = toks[t0:t0 + nt]
            n = int((np.maximum(t[:, 0], kb) >= np.minimum(t[:, 1], ke)).sum())
            count, cut, whole = count + n, cut + (n > 0 and part >= 0), whole + (n > 0 and part < 0)
    return count, cut, whole


def _check_unspoilt(x, spoilt, what):
    """The tokens that see none of the spoilt (row, key) pairs are as if there were none."""
    x.call()
    assert x.r.status() == 0
    keep = np.array([not any(s == row and a <= j < z for row, j in spoilt)
                     for s, p, a, z in R.intervals(x.b)])
    assert keep.any() and not keep.all()
    ref = R.attention(x.b, R.to64(x.q), x.k64, x.v64, 1 / np.sqrt(x.d), x.cap)
    R.assert_attention(R.to64(x.out[:x.T])[keep], tuple(r[keep] for r in ref), x.dtype, R.to64(x.lse[:x.T])[keep], what)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("heads,dtype", [((4, 4, 128), "bf16"), ((8, 8, 64), "fp16"), ((8, 8, 128), "fp16")], ids=str)
def test_later_values_of_a_cut_prompt_may_hold_anything(heads, dtype, value):
    """Tiles of a prompt cut along the keys: early tokens see nothing of the last piece,
    whose values the later tokens do see."""
    rng = np.random.default_rng(41)
    for n in (1000, 1024, 2000):
        x = Attn(R.make_batch(rng, [n], [n]), *heads, dtype)
        if n < 2000 and heads != (8, 8, 64):
            assert _empty_parts(x)[1] > 0
        for key in (200, 400, n - 1):
            _spoilt_values(x, 0, key, value)
        _check_unspoilt(x, [(0, 200), (0, 400), (0, n - 1)], f"{n} tokens")


@pytest.mark.parametrize("sms", [1, 1000])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("heads,dtype", [((8, 2, 128), "bf16"), ((14, 2, 64), "fp16")], ids=str)
def test_tokens_that_see_nothing_beside_tokens_that_see_anything(heads, dtype, value, sms):
    """In one tile: tokens with no visible key (output 0, log-sum-exp -inf), tokens of
    one document and tokens of the next, whose values hold infinities or NaN."""
    rng = np.random.default_rng(42)
    n, length = [120, 40], [900, 700]
    lo = np.repeat([0, 300], n).astype(np.int32)
    hi = np.concatenate([np.arange(z - a, z) + 1 for a, z in zip(n, length)]).astype(np.int32)
    lo[10:30], hi[10:30] = 50, 50            # nothing
    lo[30:60] = 820                          # the last document alone
    hi[60:80] = 700                          # the first alone
    lo[130:140], hi[130:140] = 5, 2          # nothing, lo past hi
    x = Attn(R.make_batch(rng, n, length, key_lo=lo, key_hi=hi), *heads, dtype, sms=sms)
    count, cut, whole = _empty_parts(x)
    assert count > 0 and (whole if sms == 1 else cut) > 0
    for s, key in ((0, 400), (0, 750), (1, 350)):
        _spoilt_values(x, s, key, value)
    _check_unspoilt(x, [(0, 400), (0, 750), (1, 350)], f"{sms} SMs")
    for t in (*range(10, 30), *range(130, 140)):
        assert not bool(x.out[t].any()) and bool((x.lse[t] == -float("inf")).all())


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("heads,dtype", [((8, 2, 128), "bf16"), ((4, 4, 64), "fp16")], ids=str)
def test_rows_that_see_nothing_of_a_shared_prefix(heads, dtype, value):
    """Rows of a group whose first visible key is behind the shared pages, beside rows
    that see an infinity or NaN there."""
    rng = np.random.default_rng(43)
    rows, pages = 24, 20
    length = [pages * 16 + int(z) for z in rng.integers(1, 60, rows)]
    lo = np.array([0 if r % 3 else pages * 16 for r in range(rows)], np.int32)
    b = R.make_batch(rng, [1] * rows, length, shared=[(range(rows), pages)], key_lo=lo,
                     group_indptr=np.array([0, rows], np.int32), group_pages=np.array([pages], np.int32))
    x = Attn(b, *heads, dtype, sms=2)
    assert x.plan.info.n_merge == rows and _empty_parts(x)[1] > 0
    _spoilt_values(x, 0, 100, value)
    _check_unspoilt(x, [(r, 100) for r in range(rows)], "group")


def test_runner_made_on_another_stream_and_called_on_the_default_one():
    """The default stream is one of the other streams to this runner: with a workspace
    of its own, zeroed before the first call there."""
    import torch
    rng = np.random.default_rng(46)
    b = R.make_batch(rng, [1, 30], [4000, 100])
    x = Attn(b, 8, 2, 128, "bf16", sms=400)
    x.run()
    want, side = x.out.clone(), torch.cuda.Stream()
    args, more = R.plan_args(b)
    with torch.cuda.stream(side):
        x.r = _runner(8, 2, 128, "bf16")
        x.r.num_sms = 400
        x.plan = x.r.plan(*args, **more)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    junk = [torch.full((1 << 18,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    del junk
    x.out.fill_(7.0)
    x.call()
    torch.cuda.synchronize()
    assert x.r.status() == 0 and torch.equal(x.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.call()
    x.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert x.r.status() == 0 and torch.equal(x.out, want)


def test_plan_made_on_another_stream_and_dropped():
    """Made on a side stream, used on the runner's first and dropped while the call waits:
    the side stream's next allocations leave the plan's memory alone."""
    import torch
    rng = np.random.default_rng(45)
    b = R.make_batch(rng, [1, 30], [400, 100])
    x = Attn(b, 8, 2, 128, "bf16")
    x.run()
    want, side = x.out.clone(), torch.cuda.Stream()
    x.out.fill_(7.0)
    args, more = R.plan_args(b)
    with torch.cuda.stream(side):
        x.plan = x.r.plan(*args, **more)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    x.call()
    at, n = x.plan.dev.data_ptr(), x.plan.dev.numel()
    del x.plan
    with torch.cuda.stream(side):
        new = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(4)]
        assert all(t.data_ptr() != at for t in new)
    torch.cuda.synchronize()
    assert x.r.status() == 0 and torch.equal(x.out, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64)], ids=str)
def test_capped_bits_do_not_depend_on_unseen_keys(heads, dtype):
    """Keys that no token sees (before its documents, past the row's end, in other
    requests' pages, what an earlier call left on the chip) change no bit, however large
    they are beside the cap; keys that only later tokens see change rounding alone."""
    import torch
    rng = np.random.default_rng(44)
    Hq, Hkv, d = heads
    n, length = [200, 37, 1, 90], [333, 700, 65, 90]
    lo = np.concatenate([[p // 64 * 64 if s == 1 else 0 for p in range(z - a, z)]
                         for s, (a, z) in enumerate(zip(n, length))]).astype(np.int32)
    for permute in (True, False):
        b = R.make_batch(rng, n, length, key_lo=lo, permute=permute, spare=20)
        x = Attn(b, Hq, Hkv, d, dtype, cap=30.0, qscale=1.0)
        ref = x.run()
        first, lse = x.out.clone(), x.lse.clone()
        other = Attn(R.make_batch(rng, [300, 1], [500, 800]), Hq, Hkv, d, dtype, cap=30.0, qscale=40.0)
        seen = {}           # (page, slot): the first token of all that sees the key
        for t, (s, p, a, z) in enumerate(R.intervals(b)):
            for j in range(a, z):
                seen.setdefault((int(b["ids"][b["ptr"][s] + j // 16]), j % 16), t)
        for trial in range(4):
            other.call()
            kc = torch.full_like(x.kc, float("nan")) if trial == 1 else x.kc * (60.0 if trial else 1.0)
            keep = 120                                     # (trial 3: the keys that later tokens see are left changed)
            for (page, slot), t in seen.items():
                if t < keep or trial < 3:
                    kc[page, :, slot] = x.kc[page, :, slot]
            x.out.fill_(7.0), x.lse.fill_(7.0)
            x.r.attend(x.plan, x.q, kc, x.vc, x.out, score_cap=x.cap, lse=x.lse)
            torch.cuda.synchronize()
            if trial < 3:
                assert torch.equal(x.out, first) and torch.equal(x.lse, lse), (permute, trial)
            else:
                R.assert_attention(R.to64(x.out[:keep]), [y[:keep] for y in ref], dtype, R.to64(x.lse[:keep]))
        assert x.r.status() == 0
