"""A small host-side driver around the C ABI: owns the RoPE table and the
workspace on one device, plans a step, copies the packed plan to the device
and enqueues the step kernel.  PyTorch is used for device memory and streams
only; all computation runs in libsarathi."""
from __future__ import annotations

import math
import threading

import numpy as np
import torch

from . import (ERR_CAPACITY, PagedArgs, PagedInfo, PlanInfo, PlanPolicy, SarathiError, Shape, _made, _stream_ptr,
               append_args, load, make_paged_batch, make_requests, paged_args, paged_calls,
               sarathi_mixed_attn, sarathi_mixed_attn_host, sarathi_paged_plan,
               sarathi_plan, sarathi_plan_bounds, sarathi_plan_ex, sarathi_rope_table,
               sarathi_shared_prefix, sarathi_workspace_status)


class StepRunner:
    def __init__(self, H_q: int, H_kv: int, d: int, max_pos: int, device="cuda", rope_theta: float = 10000.0,
                 page_size: int = 16, stream=None, rope_style: int = 0):
        self.shape = Shape(H_q, H_kv, d, page_size)
        self.device = torch.device(device)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self.num_sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.sm_scale = 1.0 / math.sqrt(d)
        self.rope_style = rope_style  # 0 rotate-half, 1 interleaved
        self.max_pos = int(max_pos)
        self.rope = torch.empty(2 * self.max_pos * d, dtype=torch.float64, device=self.device)
        sarathi_rope_table(self.rope, self.max_pos, d, rope_theta, self.stream)
        self.workspace = torch.zeros(1 << 16, dtype=torch.uint8, device=self.device)
        # the packed plan is written straight into pinned memory, so that its
        # copy to the device is one asynchronous DMA from there; PLAN_BUFFERS
        # buffers in turn, so that the host can plan up to two steps ahead of
        # the GPU without waiting
        n = self.PLAN_BUFFERS
        self._host_ts = [torch.empty(0, dtype=torch.int32) for _ in range(n)]
        self._cur = 0
        # a device copy of each: a step's plan buffers are free again once the
        # event recorded after its step call has passed
        self._plan_devs = [torch.empty(0, dtype=torch.int32, device=self.device) for _ in range(n)]
        self._upload_evts = [torch.cuda.Event() for _ in range(n)]
        self._uploaded = [False] * n  # a copy out of buffer i may be in flight (_upload_evts[i])

    PLAN_BUFFERS = 3

    def plan(self, states, prompt_len, num_computed, block_tables, budget: int, policy: PlanPolicy | None = None):
        """Plans into one of three pinned host buffers the runner keeps (taken
        in turn, grown when a batch needs more); the returned packed array is a
        view of it, valid until the next call.  The buffer's previous use
        (three plans ago) is waited for, not the last one, so a step can be
        planned while the steps before it run.  policy: a PlanPolicy
        for sarathi_plan_ex (its token_budget is used); None plans with
        sarathi_plan and `budget`."""
        reqs, keep = make_requests(states, prompt_len, num_computed, block_tables)
        return self.plan_requests(reqs, len(states), budget, policy)

    def plan_requests(self, reqs, n_reqs: int, budget: int, policy: PlanPolicy | None = None):
        """plan() from a request table the caller keeps (the ctypes array of
        make_requests, with its block tables alive; a serving loop advances it
        in place with sarathi_advance between steps)."""
        tb = policy.token_budget if policy is not None else budget
        self._cur = (self._cur + 1) % self.PLAN_BUFFERS
        c = self._cur
        if self._uploaded[c]:
            self._upload_evts[c].synchronize()  # that plan's copy has left the buffer
            self._uploaded[c] = False
        host_buf = self._host_ts[c].numpy()
        for attempt in range(2):
            try:
                if policy is not None:
                    return sarathi_plan_ex(reqs, n_reqs, policy, self.shape, self.num_sms, host_buf)
                return sarathi_plan(reqs, n_reqs, budget, self.shape, self.num_sms, host_buf)
            except SarathiError as e:
                if e.status != ERR_CAPACITY or attempt:
                    raise
                # host_buf too small, or a block table too short: size the
                # buffer by the bounds and plan again (the bounds call fails
                # the same way in the second case)
                hb, _ = sarathi_plan_bounds(reqs, n_reqs, tb, self.shape, self.num_sms)
                if host_buf.nbytes >= hb:
                    raise
                self._host_ts[c] = torch.empty(max(hb // 4 + 4, 2 * host_buf.size), dtype=torch.int32,
                                               pin_memory=True)
                host_buf = self._host_ts[c].numpy()

    def upload_plan(self, info: PlanInfo) -> torch.Tensor:
        """Enqueues on the runner's stream the copy of the packed plan of the
        last plan() call (pinned memory) into a device buffer the runner
        keeps; returns that buffer, valid until the next upload_plan."""
        n = int(info.packed_ints)
        c = self._cur
        dev = self._plan_device_buffer(n)
        # (the buffer is pinned once plan() has sized it)
        if torch.cuda.current_stream(self.device) == self.stream:
            dev[:n].copy_(self._host_ts[c][:n], non_blocking=True)
        else:
            with torch.cuda.stream(self.stream):
                dev[:n].copy_(self._host_ts[c][:n], non_blocking=True)
        self._upload_evts[c].record(self.stream)
        self._uploaded[c] = True
        return dev

    def _plan_device_buffer(self, n: int) -> torch.Tensor:
        c = self._cur
        if self._plan_devs[c].numel() < n + 4:
            torch.cuda.synchronize(self.device)  # the old buffer may be in use by an enqueued step
            self._plan_devs[c] = torch.empty(max(n + 4, 2 * self._plan_devs[c].numel()), dtype=torch.int32,
                                             device=self.device)
        return self._plan_devs[c]

    def ensure_workspace(self, nbytes: int):
        if self.workspace.numel() < nbytes:
            # rare: wait for every stream that may run a step on the old one
            torch.cuda.synchronize(self.device)
            self.workspace = torch.zeros(max(nbytes, 2 * self.workspace.numel()), dtype=torch.uint8,
                                         device=self.device)
            torch.cuda.synchronize(self.device)

    def upload(self, packed: np.ndarray) -> torch.Tensor:
        src = torch.from_numpy(np.ascontiguousarray(packed))
        dev = torch.empty(src.numel() + 4, dtype=torch.int32, device=self.device)
        dev[:src.numel()].copy_(src)
        self.stream.wait_stream(torch.cuda.current_stream(self.device))
        return dev

    def run(self, q, k, v, k_cache, v_cache, out, plan_dev: torch.Tensor, info: PlanInfo, plan_host=None) -> None:
        self.ensure_workspace(int(info.workspace_bytes))
        if info.max_kv_len > self.max_pos:
            raise ValueError(f"RoPE table covers {self.max_pos} positions, batch needs {info.max_kv_len}")
        sarathi_mixed_attn(q, k, v, k_cache, v_cache, out, plan_dev, info, self.rope, self.max_pos,
                           self.workspace, self.shape, self.sm_scale, self.stream, self.rope_style, plan_host)

    def run_planned(self, q, k, v, k_cache, v_cache, out, info: PlanInfo) -> None:
        """Enqueues the step planned by the last plan() call: one library call
        copies the packed plan from the runner's pinned buffer into its device
        buffer and launches the kernel."""
        c = self._cur
        dev = self._plan_device_buffer(int(info.packed_ints))
        self.run(q, k, v, k_cache, v_cache, out, dev, info, plan_host=self._host_ts[c])
        self._upload_evts[c].record(self.stream)
        self._uploaded[c] = True

    def run_host(self, q_host, k_host, v_host, out_host, q, k, v, k_cache, v_cache, out, info: PlanInfo,
                 stream=None, wait_event=None, done_event=None) -> None:
        """Enqueues the step planned by the last plan() call end to end from
        host buffers (one library call, sarathi_mixed_attn_host) on ``stream``
        (default: the runner's): q_host, k_host, v_host (pinned) into the
        device q, k, v, the plan into the runner's device buffer, a wait for
        ``wait_event``, the kernel, ``done_event``, out into out_host
        (pinned).  Alternating two streams, each with its own q, k, v, out
        and host buffers and the other's last done_event as wait_event,
        overlaps one step's copies and the host's planning of the next with
        the kernel before it."""
        stream = self.stream if stream is None else stream
        self.ensure_workspace(int(info.workspace_bytes))
        if info.max_kv_len > self.max_pos:
            raise ValueError(f"RoPE table covers {self.max_pos} positions, batch needs {info.max_kv_len}")
        c = self._cur
        dev = self._plan_device_buffer(int(info.packed_ints))
        sarathi_mixed_attn_host(q_host, k_host, v_host, out_host, q, k, v, k_cache, v_cache, out, dev, info,
                                self.rope, self.max_pos, self.workspace, self.shape, self.sm_scale, stream,
                                self.rope_style, self._host_ts[c], wait_event, done_event)
        self._upload_evts[c].record(stream)
        self._uploaded[c] = True

    def status(self) -> int:
        return sarathi_workspace_status(self.workspace, self.stream)


class PagedPlan:
    """A planned batch of PagedRunner: its info, and the packed plan on the device.
    Keep it while a graph that holds a call with it is replayed."""

    def __init__(self, info: PagedInfo, dev: torch.Tensor, args: PagedArgs):
        self.info, self.dev, self.args = info, dev, args
        self.home = torch.cuda.current_stream(dev.device).cuda_stream
        self.tokens, self.workspace_bytes = int(info.num_tokens), int(info.workspace_bytes)


class PagedRunner:
    """The paged operators of one attention shape on one device: owns the RoPE
    table and the workspaces, plans batches and enqueues the calls on ``stream``
    (default: the device's current stream).  dtype: the element type of every call's
    tensors, which are refused where they are of another; None: each call's own, bf16 or
    fp16.

    Calls on different streams get workspaces of their own.  Calls captured into
    CUDA graphs use the runner's main workspace, sized when a batch is planned
    (earlier, smaller ones stay alive): graphs of one runner must not be
    replayed at the same time as one another, or as its calls outside graphs on
    its first stream, and the runner has to live as long as they do."""

    def __init__(self, H_q: int, H_kv: int, d: int, dtype=None, device="cuda", max_pos: int = 0,
                 rope_theta: float = 10000.0, page_size: int = 16, rope_style: int = 0):
        self.shape = Shape(H_q, H_kv, d, page_size)
        self.dtype = dtype
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device(self.device.type, torch.cuda.current_device())
        load()
        self._calls = paged_calls()
        self.num_sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.sm_scale = 1.0 / math.sqrt(d)
        self.max_pos, self.rope_style = int(max_pos), rope_style
        self.rope = None
        if self.max_pos:
            self.rope = torch.empty(2 * self.max_pos * d, dtype=torch.float64, device=self.device)
            with torch.cuda.device(self.device):
                sarathi_rope_table(self.rope, self.max_pos, d, rope_theta, torch.cuda.current_stream(self.device))
            self._append = append_args(self.rope, self.max_pos, self.shape, rope_style)
        self._home = torch.cuda.current_stream(self.device).cuda_stream
        self._retired = []           # outgrown workspaces: captured graphs and calls in flight may hold them
        self._others = {}            # by stream
        self._lock = threading.Lock()
        self.workspace = self._zeros(1 << 16)

    def _zeros(self, nbytes: int) -> torch.Tensor:
        """A main workspace, zeroed: of the first stream's memory, whatever stream a
        batch is planned on, as that is where its calls run."""
        home = self._stream(self._home)
        with torch.cuda.stream(home):
            w = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        home.synchronize()
        return w

    def plan(self, qo_indptr, kv_page_indptr, kv_page_indices, kv_last_page_len, window: int = 0, prefix_len=None,
             key_lo=None, key_hi=None, group_indptr=None, group_pages=None, share_pages: int = 0) -> PagedPlan:
        """Plan a ragged batch (host metadata, as plan_arrays or
        sarathi_split_metadata give it) and copy the plan to the device.
        share_pages > 0: consecutive rows that share at least so many leading
        pages become groups."""
        b, keep = make_paged_batch(qo_indptr, kv_page_indptr, kv_page_indices, kv_last_page_len, window, prefix_len,
                                   key_lo, key_hi, group_indptr, group_pages)
        if share_pages:
            if group_indptr is not None:
                raise ValueError("groups or share_pages, not both")
            gi, gp = sarathi_shared_prefix(b, share_pages)
            b.n_groups, b.group_indptr, b.group_pages = len(gp), gi.ctypes.data, gp.ctypes.data
            keep += [gi, gp]
        info, packed = sarathi_paged_plan(b, self.shape, self.num_sms)
        with self._lock:
            if self.workspace.numel() < info.workspace_bytes:
                self._retired.append(self.workspace)
                self.workspace = self._zeros(max(int(info.workspace_bytes), 2 * self.workspace.numel()))
        dev = torch.from_numpy(packed).to(self.device)
        return PagedPlan(info, dev, paged_args(dev, info, self.shape, self.sm_scale))

    def _stream(self, raw: int):
        """torch's stream of a handle.  (An ExternalStream of handle 0 is a new stream
        of torch's pool, not the default stream.)"""
        return torch.cuda.ExternalStream(raw, self.device) if raw else torch.cuda.default_stream(self.device)

    def _capturing(self, raw: int, current: int) -> bool:
        """Whether stream ``raw`` is being captured (current: the current stream's handle)."""
        if raw == current and torch._C._cuda_getDevice() == self.device.index:
            return torch.cuda.is_current_stream_capturing()  # (asks the current device)
        with torch.cuda.stream(self._stream(raw)):
            return torch.cuda.is_current_stream_capturing()

    def _on(self, stream, nbytes: int):
        """The raw handle of ``stream`` (None: the current one) and the workspace of calls on it."""
        current = torch._C._cuda_getCurrentRawStream(self.device.index)
        raw = current if stream is None else _stream_ptr(stream)
        if raw == self._home:
            return raw, self.workspace
        if self._capturing(raw, current):
            return raw, self.workspace
        w = self._others.get(raw)
        if w is None or w.numel() < nbytes:
            with self._lock, torch.cuda.stream(self._stream(raw)):
                w = self._others.get(raw)
                if w is None or w.numel() < nbytes:
                    if w is not None:
                        self._retired.append(w)
                    elif self.rope is not None:
                        # (a runner dropped while its last calls run: the table, which is
                        # of the first stream's memory, is not reused before they are done)
                        self.rope.record_stream(self._stream(raw))
                    size = max(nbytes, 1 << 16, 0 if w is None else 2 * w.numel())
                    w = self._others[raw] = torch.zeros(size, dtype=torch.uint8, device=self.device)
        return raw, w

    def _typed(self, name: str, t) -> None:
        if getattr(t, "dtype", self.dtype) != self.dtype:
            raise ValueError(f"{name}: {t.dtype}, and the runner is for {self.dtype}")

    def append(self, k, v, k_cache, v_cache, slots, positions, q=None, q_out=None, sections=None, stream=None) -> None:
        """Rotate and store the new tokens' keys and values (sarathi_rope_append)."""
        if self.rope is None:
            raise ValueError("the runner has no RoPE table: give it max_pos")
        if self.dtype is not None:
            self._typed("k", k)
        raw, workspace = self._on(stream, 256)
        _made(self._calls.append, "sarathi_rope_append", self._append, self.device.index, workspace, k, v, k_cache, v_cache,
              slots, positions, q, q_out, sections, raw)

    def attend(self, plan: PagedPlan, q, k_cache, v_cache, out, score_cap: float = 0.0, slopes=None, lse=None,
               stream=None, sm_scale: float | None = None) -> None:
        """Attention of a planned batch (sarathi_paged_attn)."""
        if self.dtype is not None:
            self._typed("q", q)
        raw, workspace = self._on(stream, plan.workspace_bytes)
        if raw != plan.home and (workspace is not self.workspace or not self._capturing(
                raw, torch._C._cuda_getCurrentRawStream(self.device.index))):
            # (the plan's memory was taken on another stream: not reused before this call is
            # done.  The main workspace is that of captures and of the first stream's calls.)
            plan.dev.record_stream(self._stream(raw))
        args = plan.args
        if sm_scale is not None:
            args = PagedArgs.from_buffer_copy(args)
            args.sm_scale = sm_scale
        _made(self._calls.attend, "sarathi_paged_attn", args, self.device.index, plan.tokens, workspace, q, k_cache, v_cache,
              out, score_cap, slopes, lse, raw)

    def status(self) -> int:
        """Synchronise the device, read and clear the error words of the runner's calls (0 = fine)."""
        torch.cuda.synchronize(self.device)
        with torch.cuda.device(self.device):
            words = [sarathi_workspace_status(w) for w in (self.workspace, *self._retired, *self._others.values())]
        return next((w for w in words if w), 0)
