"""CPU tests of the paged operators' host side: the plan's work list covers every
token's visible keys once, groups and pieces among them; slots; refusals."""
import ctypes

import numpy as np
import pytest

import oracle
import workloads as W
import chunked_prefill_mixed_gb300 as S
import paged_reference as R

ITEM, TOKEN, MERGE = 8, 4, 8


def _plan(b, shape=(8, 2, 128), sms=152, host_buf=None):
    args, more = R.plan_args(b)
    share = more.pop("share_pages", 0)
    batch, keep = S.make_paged_batch(*args, **more)
    if share:
        gi, gp = S.sarathi_shared_prefix(batch, share)
        batch.n_groups, batch.group_indptr, batch.group_pages = len(gp), gi.ctypes.data, gp.ctypes.data
        keep += [gi, gp]
    return S.sarathi_paged_plan(batch, S.Shape(*shape, 16), sms, host_buf)


def _check_cover(b, shape, info, packed):
    """Every (token, kv head, visible key) in exactly one item; the partial rows of
    split tokens disjoint, and named by the token's merge record."""
    Hq, Hkv, d = shape
    G = Hq // Hkv
    iv = R.intervals(b)
    T = len(iv)
    items = packed[info.off_items:info.off_items + info.n_items * ITEM].reshape(-1, ITEM)
    toks = packed[info.off_tokens:info.off_tokens + T * TOKEN].reshape(T, TOKEN)
    merge = packed[info.off_merge:info.off_merge + info.n_merge * MERGE].reshape(-1, MERGE)
    assert info.pairs == sum(max(0, z - a) for _, _, a, z in iv)
    for t, (s, p, lo, hi) in enumerate(iv):
        assert toks[t, 2] == p and toks[t, 3] == b["ptr"][s]
        assert (toks[t, 0], toks[t, 1]) == (lo, hi) if lo < hi else toks[t, 0] >= toks[t, 1]
    seen = {}
    part_owner = np.zeros(info.n_partials, np.int64)
    direct = np.zeros((T, Hkv), np.int64)
    part_of = {}
    for n, it in enumerate(items):
        kind, g, t0, nt, kvp0, kb, ke, part = (int(x) for x in it[:8])
        assert kind == (0 if n < info.n_first else 1)
        assert kb % 16 == 0 and kb <= ke
        heads = [g]
        assert 1 <= nt <= (1 if kind else 2 * (128 // G))
        for i, h in enumerate(heads):
            if part >= 0:
                rows = np.arange(part + i * G, part + i * G + nt * G)
                assert rows[-1] < info.n_partials
                part_owner[rows] += 1
            for t in range(t0, t0 + nt):
                own = b["ids"][int(toks[t, 3]):][:max(1, -(-ke // 16))]
                assert np.array_equal(own[kb // 16:], b["ids"][kvp0:][:len(own)][kb // 16:]), "the item's pages"
                if part < 0:
                    direct[t, h] += 1
                else:
                    part_of.setdefault((t, h), set()).add(part + i * G + (t - t0) * G)
                a, z = max(kb, int(toks[t, 0])), min(ke, int(toks[t, 1]))
                if a < z:
                    seen.setdefault((t, h), []).append((a, z))
    assert np.all(part_owner == 1)
    for t, (s, p, lo, hi) in enumerate(iv):
        for h in range(Hkv):
            got = sorted(seen.get((t, h), []))
            assert all(x[1] == y[0] for x, y in zip(got, got[1:])), "gap or overlap"
            if lo < hi:
                assert got[0][0] == lo and got[-1][1] == hi
            else:
                assert not got
    merged = set(int(m[0]) for m in merge)
    assert len(merged) == len(merge)
    for m in merge:
        for h in range(Hkv):
            named = set()
            for n, base, step in (m[1:4], m[4:7]):
                named |= {int(base + (k * Hkv + h) * step) for k in range(n)}
            assert named == part_of.get((int(m[0]), h), set())
    for t in range(T):
        assert np.all(direct[t] == (0 if t in merged else 1))


@pytest.mark.parametrize("sms", [1, 152, 2000])
@pytest.mark.parametrize("shape", [(8, 2, 128), (4, 4, 64), (14, 2, 128), (3, 3, 64), (16, 1, 128)], ids=str)
def test_work_list_covers_every_visible_key_once(shape, sms):
    rng = np.random.default_rng(shape[0] + sms)
    for trial in range(25):
        R_ = int(rng.integers(1, 7))
        n = [int(rng.choice([0, 1, 1, 2, 17, 130, 300])) for _ in range(R_)]
        length = [max(1, x + int(rng.choice([0, 0, 5, 100, 1500, 6000]))) for x in n]
        b = R.make_batch(rng, n, length)
        T = sum(n)
        kind = trial % 5
        if kind == 1:
            b["window"] = int(rng.integers(1, 400))
        elif kind == 2:
            b["prefix_len"] = rng.integers(0, 500, R_).astype(np.int32)
        elif kind == 3:
            b["key_lo"] = rng.integers(-3, 400, T).astype(np.int32)
        elif kind == 4:
            b["key_lo"], b["key_hi"] = (rng.integers(-3, 900, T).astype(np.int32) for _ in range(2))
        info, packed = _plan(b, shape, sms)
        _check_cover(b, shape, info, packed)


@pytest.mark.parametrize("sms", [1, 152, 2000])
def test_groups_cover_every_visible_key_once(sms):
    rng = np.random.default_rng(sms)
    for trial in range(20):
        pages = int(rng.integers(1, 60))
        rows = int(rng.integers(2, 40))
        length = [pages * 16 + int(rng.integers(0, 200)) for _ in range(rows)] + [50, 700]
        n = [int(rng.choice([1, 1, 1, 4])) for _ in range(rows)] + [1, 70]
        b = R.make_batch(rng, n, length, shared=[(range(rows), pages)],
                         group_indptr=np.array([0, rows, rows + 2], np.int32), group_pages=np.array([pages, 0], np.int32))
        if trial % 2:
            b["window"] = int(rng.integers(1, 2000))
        info, packed = _plan(b, (8, 2, 128), sms)
        _check_cover(b, (8, 2, 128), info, packed)


@pytest.mark.parametrize("heads,rows,pages,grouped", [((32, 8, 128), 64, 4, False), ((32, 8, 128), 64, 16, True),
                                                     ((32, 8, 128), 2, 64, False), ((64, 8, 64), 2, 16, False),
                                                     ((64, 8, 64), 8, 256, True)])
def test_small_groups_are_left_to_their_rows(heads, rows, pages, grouped):
    b = R.make_batch(np.random.default_rng(7), [1] * rows, [16 * pages + 9] * rows, shared=[(range(rows), pages)],
                     share_pages=1)
    info, packed = _plan(b, heads)
    assert (info.n_first > 0) == grouped
    _check_cover(b, heads, info, packed)
    # rows of several tokens are tiles anyway
    b = R.make_batch(np.random.default_rng(7), [2] + [1] * rows, [16 * pages + 9] * (rows + 1),
                     shared=[(range(rows + 1), pages)], share_pages=1)
    info, packed = _plan(b, heads)
    assert info.n_first > 0 and info.n_merge == rows + 2
    _check_cover(b, heads, info, packed)


def test_shared_prefix_finds_the_runs():
    rng = np.random.default_rng(5)
    b = R.make_batch(rng, [1] * 7, [100, 100, 200, 64, 64, 33, 33],
                     shared=[((0, 1, 2), 5), ((3, 4), 4)])
    b["ids"][b["ptr"][5]:b["ptr"][5] + 2] = [3, 4]
    b["ids"][b["ptr"][6]:b["ptr"][6] + 2] = [3, 5]
    args, _ = R.plan_args(b)
    batch, keep = S.make_paged_batch(*args)
    gi, gp = S.sarathi_shared_prefix(batch, 1)
    # (64 keys, the last of them new: three whole pages before it)
    assert gi.tolist() == [0, 3, 5, 7] and gp.tolist() == [5, 3, 1]
    gi, gp = S.sarathi_shared_prefix(batch, 4)
    assert gi.tolist() == [0, 3, 4, 5, 6, 7] and gp.tolist() == [5, 0, 0, 0, 0]
    with pytest.raises(S.SarathiError):
        S.sarathi_shared_prefix(batch, 0)
    empty, keep2 = S.make_paged_batch([0], [0], [], [])
    gi, gp = S.sarathi_shared_prefix(empty, 1)
    assert gi.tolist() == [0] and gp.size == 0


def test_slot_mapping_names_the_plan_tokens_slots():
    wl = W.tiny(1)
    reqs, keep = S.make_requests(*wl.arrays())
    st, info, packed = S.sarathi_plan(reqs, len(wl.requests), wl.budget, S.Shape(4, 4, 64, 16), 152)
    slots, pos = S.sarathi_slot_mapping(info, packed)
    m = S.plan_arrays(info, packed)
    t = 0
    for s in range(m["n_sched"]):
        n = m["qo_indptr"][s + 1] - m["qo_indptr"][s]
        ids = m["kv_page_indices"][m["kv_page_indptr"][s]:m["kv_page_indptr"][s + 1]]
        kv = (len(ids) - 1) * 16 + m["kv_last_page_len"][s]
        for p in range(kv - n, kv):
            assert pos[t] == p and slots[t] == ids[p // 16] * 16 + p % 16
            t += 1
    assert t == info.num_tokens == len(slots)
    assert S.load().sarathi_slot_mapping(None, None, None, None) == S.ERR_INVALID_ARG


def test_streams_are_split_where_that_shortens_them():
    rng = np.random.default_rng(8)
    for rows, pages, split in ((150, 6, False), (1, 20, True), (64, 4, False), (4, 300, True)):
        b = R.make_batch(rng, [1] * rows, [16 * pages] * rows)
        info, packed = _plan(b, (32, 8, 128))
        assert info.n_merge == (rows if split else 0), (rows, pages)
        _check_cover(b, (32, 8, 128), info, packed)


@pytest.mark.parametrize("sms", [1, 152])
def test_pieces_of_long_rows_are_bounded(sms):
    b = R.make_batch(np.random.default_rng(3), [300, 1], [300000, 70000])
    info, packed = _plan(b, (8, 2, 64), sms)
    items = packed[info.off_items:info.off_items + ITEM * info.n_items].reshape(-1, ITEM)
    tiles = items[items[:, 0] == 0]
    assert (tiles[:, 6] - tiles[:, 5]).max() <= 1 << 17
    for g in range(2):   # each tile's pieces follow one another over all the keys that it sees
        for t0 in np.unique(tiles[:, 2]):
            p = tiles[(tiles[:, 1] == g) & (tiles[:, 2] == t0)]
            p = p[np.argsort(p[:, 5])]
            assert p[0, 5] == 0 and (p[1:, 5] == p[:-1, 6]).all() and p[-1, 6] >= 299700 + t0 + 1


def test_empty_batches():
    info, packed = _plan(R.make_batch(np.random.default_rng(0), [0, 0], [30, 40]))
    assert info.num_tokens == 0 and info.n_items == 0
    batch, keep = S.make_paged_batch([0], [0], [], [])
    info, packed = S.sarathi_paged_plan(batch, S.Shape(8, 2, 128, 16), 152)
    assert info.num_tokens == 0 and info.n_items == 0 and info.workspace_bytes >= 256


def _good():
    return R.make_batch(np.random.default_rng(1), [1, 20, 1], [100, 64, 100], shared=[((0, 2), 3)])


def test_plan_refusals():
    ok = S.Shape(8, 2, 128, 16)

    def status(shape=ok, sms=152, **change):
        b = _good()
        args, more = R.plan_args(b)
        batch, keep = S.make_paged_batch(*args)
        for k, v in change.items():
            if isinstance(v, np.ndarray):
                keep.append(v)
                v = v.ctypes.data
            setattr(batch, k, v)
        try:
            S.sarathi_paged_plan(batch, shape, sms)
            return S.OK
        except S.SarathiError as e:
            return e.status
    i32 = lambda *x: np.array(x, np.int32)  # noqa: E731
    assert status() == S.OK
    for change in (dict(n_rows=-1), dict(qo_indptr=None), dict(kv_page_indptr=None), dict(kv_page_indices=None),
                   dict(kv_last_page_len=None), dict(qo_indptr=i32(1, 2, 22, 23)), dict(qo_indptr=i32(0, 2, 1, 3)),
                   dict(kv_page_indptr=i32(0, 7, 5, 18)), dict(kv_last_page_len=i32(0, 16, 4)),
                   dict(kv_last_page_len=i32(4, 17, 4)), dict(qo_indptr=i32(0, 1, 66, 67)),
                   dict(kv_page_indptr=i32(0, 0, 4, 11)), dict(window=-1), dict(prefix_len=i32(0, -1, 0)),
                   dict(n_groups=-1), dict(n_groups=1), dict(n_groups=1, group_indptr=i32(0, 3), group_pages=i32(-1)),
                   dict(n_groups=1, group_indptr=i32(0, 4), group_pages=i32(0)),
                   dict(n_groups=1, group_indptr=i32(-1, 2), group_pages=i32(0)),
                   dict(n_groups=1, group_indptr=i32(0, 2), group_pages=i32(1)),
                   dict(n_groups=1, group_indptr=i32(0, 1), group_pages=i32(7))):
        assert status(**change) == S.ERR_INVALID_ARG, change
    assert status(sms=0) == S.ERR_INVALID_ARG
    assert status(shape=S.Shape(8, 3, 128, 16)) == S.ERR_INVALID_ARG
    for shape in (S.Shape(8, 2, 96, 16), S.Shape(8, 2, 128, 32), S.Shape(34, 2, 128, 16)):
        assert status(shape=shape) == S.ERR_UNSUPPORTED
    # a buffer too small: the size that is needed
    args, _ = R.plan_args(_good())
    batch, keep = S.make_paged_batch(*args)
    info, buf = S.PagedInfo(), np.zeros(8, np.int32)
    st = S.load().sarathi_paged_plan(ctypes.byref(batch), ctypes.byref(ok), 152, buf.ctypes.data, buf.nbytes,
                                     ctypes.byref(info))
    assert st == S.ERR_CAPACITY and info.packed_ints > 8 and not buf.any()
    # (the Python side's own)
    for bad in (dict(prefix_len=[1]), dict(key_lo=[1]), dict(key_hi=np.zeros(50)), dict(group_pages=[1]),
                dict(group_indptr=[0, 1, 2], group_pages=[1])):
        with pytest.raises(ValueError):
            S.make_paged_batch(*args, **bad)
    with pytest.raises(ValueError):
        S.make_paged_batch([0, 1], [0], [], [])


def test_call_refusals_before_any_launch():
    """Status codes of the two device calls on arguments that they refuse: nothing
    is enqueued, so no GPU is needed."""
    lib = S.load()
    shape = S.Shape(8, 2, 128, 16)

    def append(**change):
        a = S.AppendArgs(q=0x1000, q_out=0x1000, k=0x1000, v=0x1000, q_stride=1024, q_out_stride=1024, k_stride=256,
                         v_stride=256, k_cache=0x1000, v_cache=0x1000, slots=0x1000, positions=0x1000, tokens=0,
                         n_axes=1, rope_table=0x1000, rope_max_pos=10, num_pages=4, dtype=S.BF16, shape=shape,
                         workspace=0x1000)
        a.sections[0] = 64
        for k, v in change.items():
            if k == "sections":
                for i, x in enumerate(v):
                    a.sections[i] = x
            else:
                setattr(a, k, v)
        return lib.sarathi_rope_append(ctypes.byref(a), None)
    assert lib.sarathi_rope_append(None, None) == S.ERR_INVALID_ARG
    assert append() == S.OK   # no tokens: nothing to do
    for change in (dict(tokens=-1), dict(rope_style=2), dict(n_axes=0), dict(n_axes=5), dict(sections=(63,)),
                   dict(n_axes=2, sections=(60, 3)), dict(n_axes=2, sections=(70, -6)), dict(rope_max_pos=0),
                   dict(num_pages=0)):
        assert append(**change) == S.ERR_INVALID_ARG, change
    for change in (dict(k=None), dict(v=None), dict(k_cache=None), dict(v_cache=None), dict(slots=None),
                   dict(positions=None), dict(rope_table=None), dict(workspace=None), dict(q=None), dict(q_out=None),
                   dict(q=0x1008), dict(k=0x1004), dict(v=0x1002), dict(k_cache=0x1008), dict(q_out=0x1008),
                   dict(slots=0x1001), dict(workspace=0x1010), dict(k_stride=255), dict(k_stride=260),
                   dict(v_stride=128), dict(q_stride=1000), dict(q_out_stride=1028),
                   dict(q_out_stride=2048)):
        assert append(tokens=3, **change) == S.ERR_INVALID_ARG, change
    assert append(dtype=2) == S.ERR_UNSUPPORTED
    assert append(num_pages=1 << 27) == S.ERR_UNSUPPORTED

    info, packed = _plan(_good())

    def attend(**change):
        a = S.PagedArgs(q=0x1000, q_stride=1024, k_cache=0x1000, v_cache=0x1000, out=0x10000000, plan=0x1000,
                        info=ctypes.pointer(info), num_pages=100, dtype=S.BF16, workspace=0x1000,
                        workspace_bytes=1 << 40, shape=shape, sm_scale=0.1, score_cap=0.0)
        for k, v in change.items():
            setattr(a, k, v)
        return lib.sarathi_paged_attn(ctypes.byref(a), None)
    assert lib.sarathi_paged_attn(None, None) == S.ERR_INVALID_ARG
    nan, inf = float("nan"), float("inf")
    for change in (dict(info=None), dict(q=None), dict(k_cache=None), dict(v_cache=None), dict(out=None),
                   dict(plan=None), dict(workspace=None), dict(q=0x1008), dict(out=0x1004), dict(plan=0x1004),
                   dict(lse=0x1002), dict(slopes=0x1001), dict(workspace=0x1080), dict(q_stride=1000),
                   dict(q_stride=1028), dict(sm_scale=0.0), dict(sm_scale=nan), dict(sm_scale=-1.0),
                   dict(sm_scale=inf), dict(score_cap=-1.0), dict(score_cap=nan), dict(score_cap=inf),
                   dict(sm_scale=1e-40), dict(sm_scale=3e38), dict(score_cap=3e38), dict(score_cap=1e-39),
                   dict(sm_scale=1e-30, score_cap=1e30), dict(sm_scale=1e10, score_cap=1e-30),
                   dict(q=0x10000000), dict(out=0x1000 + 2048 * info.num_tokens - 16), dict(out=0x1000 - 16),
                   dict(num_pages=0), dict(shape=S.Shape(8, 4, 128, 16))):
        assert attend(**change) == S.ERR_INVALID_ARG, change
    assert attend(workspace_bytes=info.workspace_bytes - 1) == S.ERR_CAPACITY
    assert attend(dtype=7) == S.ERR_UNSUPPORTED
    assert attend(num_pages=1 << 27) == S.ERR_UNSUPPORTED


def test_python_refusals():
    """Tensors that do not fit are refused before the library is called."""
    import torch
    shape = S.Shape(8, 2, 64, 16)
    bf = dict(dtype=torch.bfloat16)
    k, q = torch.zeros(5, 2, 64, **bf), torch.zeros(5, 8, 64, **bf)
    pool, slots = torch.zeros(3, 2, 16, 64, **bf), torch.zeros(5, dtype=torch.int32)
    table, ws = torch.zeros(2 * 10 * 64, dtype=torch.float64), torch.zeros(256, dtype=torch.uint8)

    def append(**change):
        a = dict(k=k, v=k, k_cache=pool, v_cache=pool, slots=slots, positions=slots, rope_table=table,
                 rope_max_pos=10, shape=shape, workspace=ws, q=q, q_out=q)
        a.update(change)
        S.sarathi_rope_append(**a)
    for change in (dict(k=k.float()), dict(v=k.half()), dict(k=k[:, :1]), dict(v=k[:4]), dict(k_cache=pool[:, :1]),
                   dict(v_cache=pool[:2]), dict(k_cache=pool.transpose(0, 1)), dict(slots=slots.long()),
                   dict(slots=slots[:4]), dict(positions=slots.float()), dict(sections=(16, 16)),
                   dict(sections=(7, 7, 7, 7, 4)), dict(rope_table=table[:-1]), dict(q=None), dict(q=q[:, ::2]),
                   dict(q_out=q[..., :32]), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)),
                   dict(workspace=ws[:100]), dict(k=None), dict(v=[1.0]), dict(sections=()), dict(sections=(-1, 33)),
                   dict(sections=(2 ** 33, 0)), dict(sections=(16, 16), positions=torch.zeros(10, dtype=torch.int32)),
                   dict(k_cache=pool.float()), dict(q=q.half(), q_out=q.half()), dict(q_out=None), dict(slots=None),
                   dict(k=k[0]), {}):   # (as it stands: CPU tensors)
        with pytest.raises(ValueError):
            append(**change)
    b = R.make_batch(np.random.default_rng(1), [5], [5])
    info, packed = _plan(b, (8, 2, 64))
    plan = torch.zeros(info.packed_ints, dtype=torch.int32)
    big = torch.zeros(1 << 16, dtype=torch.uint8)

    def attend(**change):
        a = dict(q=q, k_cache=pool, v_cache=pool, out=q.clone(), plan_dev=plan, info=info, workspace=big, shape=shape,
                 sm_scale=0.1)
        a.update(change)
        S.sarathi_paged_attn(**a)
    for change in (dict(q=q[:4]), dict(q=q.float()), dict(out=q[:4]), dict(out=q.half()), dict(k_cache=pool.half()),
                   dict(v_cache=pool[:1]), dict(plan_dev=plan[:-1]), dict(plan_dev=plan.long()),
                   dict(slopes=torch.zeros(8, dtype=torch.float64)), dict(slopes=torch.zeros(7)),
                   dict(lse=torch.zeros(4, 8)), dict(lse=torch.zeros(5, 8, dtype=torch.float64)), dict(q=None), dict(out=None),
                   dict(slopes=1.0), dict(lse=torch.zeros(5, 16)[:, ::2]), dict(workspace=None), dict(q=q[:, :, ::2]), {}):
        with pytest.raises(ValueError):
            attend(**change)
    good = dict(qo_indptr=[0, 5], kv_page_indptr=[0, 1], kv_page_indices=[0], kv_last_page_len=[5])
    S.make_paged_batch(**good, key_hi=np.full(5, 2 ** 31 - 1))
    for change in (dict(key_hi=np.full(5, 2 ** 31)), dict(key_lo=np.full(5, -2 ** 31 - 1)),
                   dict(kv_page_indices=[2 ** 40]), dict(key_hi=np.zeros(5)), dict(key_hi=[3] * 4),
                   dict(kv_last_page_len=[5, 5]), dict(group_pages=[1])):
        with pytest.raises(ValueError):
            S.make_paged_batch(**dict(good, **change))


def _attend_on_cpu(**change):
    """sarathi_paged_attn on CPU tensors, which it refuses at the end where nothing else is wrong."""
    import torch
    b = R.make_batch(np.random.default_rng(1), [5], [5])
    info, packed = _plan(b, (8, 2, 64))
    q, pool = torch.zeros(5, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    a = dict(q=q, k_cache=pool, v_cache=pool, out=q.clone(), plan_dev=torch.zeros(info.packed_ints, dtype=torch.int32),
             info=info, workspace=torch.zeros(1 << 16, dtype=torch.uint8), shape=S.Shape(8, 2, 64, 16), sm_scale=0.1)
    a.update(change)
    S.sarathi_paged_attn(**a)


def test_a_cap_too_small_for_fp32_is_refused():
    """Rounded to 0 it would stand for no cap."""
    for cap in (1e-50, -1e-50, 1e-320):
        with pytest.raises(ValueError, match="score_cap"):
            _attend_on_cpu(score_cap=cap)
    for cap in (0.0, -0.0, 1e-30, 50):
        with pytest.raises(ValueError, match="CUDA device"):
            _attend_on_cpu(score_cap=cap)


def test_a_window_or_page_count_outside_int32_is_refused():
    """They would wrap: a window of 2^32 + 3 keys to one of 3."""
    good = dict(qo_indptr=[0, 5], kv_page_indptr=[0, 1], kv_page_indices=[0], kv_last_page_len=[5])
    for window in (2 ** 31, 2 ** 32 + 3, -2 ** 32 + 3):
        with pytest.raises(ValueError, match="window"):
            S.make_paged_batch(**good, window=window)
    batch, keep = S.make_paged_batch(**good, window=2 ** 31 - 1)
    assert batch.window == 2 ** 31 - 1
    info, packed = S.sarathi_paged_plan(batch, S.Shape(8, 2, 128, 16), 152)
    assert info.pairs == 15
    for pages in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="min_pages"):
            S.sarathi_shared_prefix(batch, pages)


def test_a_buffer_that_cannot_hold_a_plan_as_int32_is_refused():
    """Its words would be read as other numbers, or from between them."""
    args, _ = R.plan_args(_good())
    batch, keep = S.make_paged_batch(*args)
    shape, fixed = S.Shape(8, 2, 128, 16), np.zeros(1 << 14, np.int32)
    fixed.flags.writeable = False
    for buf in (np.zeros(1 << 14, np.int64), np.zeros(1 << 14, np.int32)[::2], np.zeros((2, 1 << 13), np.int32), fixed,
                np.zeros(1 << 14, np.uint8)):
        with pytest.raises(ValueError, match="host_buf"):
            S.sarathi_paged_plan(batch, shape, 152, buf)
        assert not buf.any()
    want = S.sarathi_paged_plan(batch, shape, 152)[1]
    for n in (8, 1 << 14):      # (too small: a larger one is taken)
        assert np.array_equal(S.sarathi_paged_plan(batch, shape, 152, np.zeros(n, np.int32))[1], want)


def test_a_workspace_of_fewer_bytes_than_elements_is_refused():
    """An expanded tensor has many elements in a few bytes of memory: the kernels would
    write past them."""
    import torch
    one = torch.zeros(1, dtype=torch.uint8)
    for ws in (one.expand(1 << 16), torch.zeros(1 << 17, dtype=torch.uint8)[::2], one.expand(256, 256)):
        with pytest.raises(ValueError, match="workspace"):
            _attend_on_cpu(workspace=ws)
        k, pool = torch.zeros(5, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
        slots = torch.zeros(5, dtype=torch.int32)
        with pytest.raises(ValueError, match="workspace"):
            S.sarathi_rope_append(k, k, pool, pool, slots, slots, torch.zeros(2 * 10 * 64, dtype=torch.float64), 10,
                                  S.Shape(8, 2, 64, 16), ws)
