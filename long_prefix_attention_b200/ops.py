"""Python binding of the ASM C ABI (include/asm.h) for torch CUDA tensors.

Each function has the name of the C entry point it calls and only marshals
arguments: shapes are read from the tensors, pointers and the current CUDA
stream are passed through, and a non-OK status raises :class:`AsmError`.
Every computation runs in the library's sm_100a kernels; outputs are written
into the tensors the caller passes.  The ``alloc_*`` helpers only allocate
correctly sized (and, for decode workspaces, zeroed) buffers.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

ASM_OK, ASM_ERR_INVALID_ARG, ASM_ERR_UNSUPPORTED, ASM_ERR_WORKSPACE, ASM_ERR_CUDA, ASM_ERR_TIMEOUT = range(6)
ASM_F32, ASM_BF16 = 0, 1
ASM_L2, ASM_COSINE = 0, 1
ASM_ZBAR_MEAN, ASM_ZBAR_SUM = 0, 1
ASM_DECODE_PREFETCH_CENTROIDS = 1
ASM_ROPE_HALF, ASM_ROPE_PAIRS = 0, 1
(ASM_ROPE_SCALE_NONE, ASM_ROPE_SCALE_LINEAR, ASM_ROPE_SCALE_BASE, ASM_ROPE_SCALE_BANDS,
 ASM_ROPE_SCALE_YARN) = range(5)

_DT = {torch.float32: ASM_F32, torch.bfloat16: ASM_BF16}


class AsmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib = _lib.load()
        msg = lib.asm_status_string(status).decode()
        if status == ASM_ERR_CUDA:
            msg += ": " + lib.asm_last_cuda_error().decode()
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise AsmError(fn, status)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"storage dtype must be float32 or bfloat16, got {t.dtype}")
    return _DT[t.dtype]


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def status_string(status: int) -> str:
    return _lib.load().asm_status_string(int(status)).decode()


def version() -> str:
    return _lib.load().asm_version().decode()


# ------------------------------------------------------------------ build --

def asm_build_states(q, k, v, scale: float, a, logz, accumulate: bool = False, stream=None):
    """States of q[Hq,N,d] over the prefix block k,v[Hkv,L,d] into a, logz."""
    _contig(q, k, v, a, logz)
    Hq, N, d = q.shape
    Hkv, L, _ = k.shape
    _check("asm_build_states", _lib.load().asm_build_states(
        _p(q), _p(k), _p(v), Hq, Hkv, N, L, d, float(scale), _dt(q), int(bool(accumulate)),
        _p(a), _p(logz), _stream(stream)))


def asm_merge_states(a_acc, logz_acc, a_in, logz_in, stream=None):
    """Fold the states (a_in, logz_in) into (a_acc, logz_acc) by the
    online-softmax identity, row by row (any leading shape, d innermost)."""
    _contig(a_acc, logz_acc, a_in, logz_in)
    if a_acc.shape != a_in.shape or logz_acc.shape != logz_in.shape or a_acc.dtype != a_in.dtype:
        raise AsmError("asm_merge_states", ASM_ERR_INVALID_ARG)
    d = a_acc.shape[-1]
    R = a_acc.numel() // d
    if logz_acc.numel() != R:
        raise AsmError("asm_merge_states", ASM_ERR_INVALID_ARG)
    _check("asm_merge_states", _lib.load().asm_merge_states(
        _p(a_acc), _p(logz_acc), _p(a_in), _p(logz_in), R, d, _dt(a_acc), _stream(stream)))


def asm_kmeanspp_workspace_size(H: int, N: int, d: int, K: int) -> int:
    return int(_lib.load().asm_kmeanspp_workspace_size(H, N, d, K))


def asm_kmeanspp_seed(x, u, init_idx, ws, stream=None):
    """k-means++ indices init_idx[H,K] of x[H,N,d] from the draws u[H,K] (fp64)."""
    _contig(x, u, init_idx)
    H, N, d = x.shape
    K = u.shape[1]
    _check("asm_kmeanspp_seed", _lib.load().asm_kmeanspp_seed(
        _p(x), H, N, d, K, _p(u), _dt(x), _p(init_idx), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def asm_kmeanspp_batched_workspace_size(H: int, N: int, d: int, K: int, batch: int) -> int:
    return int(_lib.load().asm_kmeanspp_batched_workspace_size(H, N, d, K, batch))


def asm_kmeanspp_seed_batched(x, u, init_idx, batch: int, ws, stream=None):
    """Batched k-means++ indices init_idx[H,K] of x[H,N,d]: up to `batch`
    draws per round from the same D2 distribution, draws u[H,U] (fp64) used
    in order."""
    _contig(x, u, init_idx)
    H, N, d = x.shape
    K = init_idx.shape[1]
    _check("asm_kmeanspp_seed_batched", _lib.load().asm_kmeanspp_seed_batched(
        _p(x), H, N, d, K, int(batch), _p(u), u.shape[1], _dt(x), _p(init_idx), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def asm_kmeans_workspace_size(H: int, N: int, d: int, K: int) -> int:
    return int(_lib.load().asm_kmeans_workspace_size(H, N, d, K))


def asm_kmeans_assign(x, centroids_dt, assign, ws, metric: int = ASM_L2, stream=None):
    _contig(x, centroids_dt, assign)
    H, N, d = x.shape
    K = centroids_dt.shape[1]
    _check("asm_kmeans_assign", _lib.load().asm_kmeans_assign(
        _p(x), _p(centroids_dt), H, N, d, K, int(metric), _dt(x), _p(assign), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def asm_kmeans_update(x, assign, centroids, centroids_dt, counts, perm, seg_off, ws, stream=None):
    _contig(x, assign, centroids, centroids_dt, counts, perm, seg_off)
    H, N, d = x.shape
    K = centroids.shape[1]
    _check("asm_kmeans_update", _lib.load().asm_kmeans_update(
        _p(x), _p(assign), H, N, d, K, _dt(x), _p(centroids), _p(centroids_dt), _p(counts),
        _p(perm), _p(seg_off), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def asm_kmeans(x, init_idx, iters: int, centroids, centroids_dt, assign, counts, perm, seg_off,
               ws, metric: int = ASM_L2, stream=None):
    _contig(x, init_idx, centroids, centroids_dt, assign, counts, perm, seg_off)
    H, N, d = x.shape
    K = init_idx.shape[1]
    _check("asm_kmeans", _lib.load().asm_kmeans(
        _p(x), H, N, d, K, int(iters), int(metric), _dt(x), _p(init_idx), _p(centroids),
        _p(centroids_dt), _p(assign), _p(counts), _p(perm), _p(seg_off), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def asm_aggregate(a, logz, perm, seg_off, a_bar, logz_bar, zmode: int = ASM_ZBAR_MEAN,
                  stream=None):
    _contig(a, logz, perm, seg_off, a_bar, logz_bar)
    H, N, d = a.shape
    K = a_bar.shape[1]
    _check("asm_aggregate", _lib.load().asm_aggregate(
        _p(a), _p(logz), _p(perm), _p(seg_off), H, N, d, K, int(zmode), _dt(a), _p(a_bar),
        _p(logz_bar), _stream(stream)))


# ----------------------------------------------------------------- decode --

def asm_decode_workspace_size(B, Hq, Hkv, K, Tmax, d, dtype) -> int:
    return int(_lib.load().asm_decode_workspace_size(B, Hq, Hkv, K, Tmax, d, _DT[dtype]))


def asm_decode_step_launches(B, Hq, Hkv, K, Tmax, d, dtype) -> int:
    """Kernel launches of one asm_decode_step with these sizes on the current device."""
    return int(_lib.load().asm_decode_step_launches(B, Hq, Hkv, K, Tmax, d, _DT[dtype]))


def asm_flash_decode_workspace_size(B, Hq, Hkv, Lp, Tmax, d, dtype) -> int:
    return int(_lib.load().asm_flash_decode_workspace_size(B, Hq, Hkv, Lp, Tmax, d, _DT[dtype]))


def asm_workspace_init(ws, stream=None):
    _check("asm_workspace_init", _lib.load().asm_workspace_init(
        _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def asm_workspace_error(ws, stream=None) -> int:
    code = ctypes.c_int(0)
    _check("asm_workspace_error", _lib.load().asm_workspace_error(
        _p(ws), ws.numel() * ws.element_size(), ctypes.byref(code), _stream(stream)))
    return code.value


def asm_wait_spin_limit() -> int:
    """Unsuccessful try_wait polls after which any library wait gives up."""
    return int(_lib.load().asm_wait_spin_limit())


def asm_wait_selftest(polls: int, ws, stream=None) -> int:
    """Run a bounded wait that nothing completes (polls try_wait polls, 0 =
    the library's own bound); returns its duration in ns.  The workspace's
    error word then holds ASM_ERR_TIMEOUT (read with asm_workspace_error)."""
    ns = ctypes.c_uint64(0)
    _check("asm_wait_selftest", _lib.load().asm_wait_selftest(
        int(polls), _p(ws), ws.numel() * ws.element_size(), ctypes.byref(ns), _stream(stream)))
    return int(ns.value)


def asm_decode_step(q, centroids, a_bar, logz_bar, k_cache, v_cache, local_len, scale: float,
                    out, ws, lse_out=None, idx_out=None, metric: int = ASM_L2, flags: int = 0,
                    stream=None):
    """One decode step: lookup + merge with local attention, into out[B,Hq,d]."""
    _contig(q, centroids, a_bar, logz_bar, k_cache, v_cache, local_len, out, lse_out, idx_out)
    B, Hq, d = q.shape
    K = centroids.shape[1]
    _, Hkv, Tmax, _ = k_cache.shape
    _check("asm_decode_step", _lib.load().asm_decode_step(
        _p(q), _p(centroids), _p(a_bar), _p(logz_bar), _p(k_cache), _p(v_cache), _p(local_len),
        B, Hq, Hkv, K, Tmax, d, float(scale), int(metric), _dt(q), _p(out), _p(lse_out),
        _p(idx_out), int(flags), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def asm_decode_step_search(q, q_search, centroids, a_bar, logz_bar, k_cache, v_cache, local_len,
                           scale: float, out, ws, lse_out=None, idx_out=None, metric: int = ASM_L2,
                           flags: int = 0, stream=None):
    """asm_decode_step whose centroid search uses q_search[B,Hq,d] (e.g. the
    whitened queries) while the local attention and the merge use q."""
    _contig(q, q_search, centroids, a_bar, logz_bar, k_cache, v_cache, local_len, out, lse_out, idx_out)
    if q_search.shape != q.shape or q_search.dtype != q.dtype:
        raise AsmError("asm_decode_step_search", ASM_ERR_INVALID_ARG)
    B, Hq, d = q.shape
    K = centroids.shape[1]
    _, Hkv, Tmax, _ = k_cache.shape
    _check("asm_decode_step_search", _lib.load().asm_decode_step_search(
        _p(q), _p(q_search), _p(centroids), _p(a_bar), _p(logz_bar), _p(k_cache), _p(v_cache),
        _p(local_len), B, Hq, Hkv, K, Tmax, d, float(scale), int(metric), _dt(q), _p(out), _p(lse_out),
        _p(idx_out), int(flags), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def asm_whitening_workspace_size(H: int, d: int) -> int:
    return int(_lib.load().asm_whitening_workspace_size(H, d))


def asm_whitening(x, mu, W, ws, eps_rel: float = 1e-5, stream=None):
    """ZCA whitening of each head of x[H,N,d]: mu[H,d] and W[H,d,d] (fp32)."""
    _contig(x, mu, W)
    H, N, d = x.shape
    _check("asm_whitening", _lib.load().asm_whitening(
        _p(x), H, N, d, _dt(x), float(eps_rel), _p(mu), _p(W), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def asm_whiten(x, mu, W, y, layout: str | None = None, stream=None):
    """y = W[h] (x - mu[h]) row by row.  layout "heads": x, y are [H, R, d]
    (calibration points, centres); "batch": [R, H, d] (decode queries).  When
    omitted it is inferred from which dimension equals H = mu.shape[0], and
    must then be unambiguous."""
    _contig(x, mu, W, y)
    H, d = mu.shape
    if x.shape != y.shape or x.dtype != y.dtype or x.dim() != 3 or x.shape[2] != d:
        raise AsmError("asm_whiten", ASM_ERR_INVALID_ARG)
    if layout is None:
        if (x.shape[0] == H) == (x.shape[1] == H):
            raise AsmError("asm_whiten", ASM_ERR_INVALID_ARG)
        layout = "heads" if x.shape[0] == H else "batch"
    if layout == "heads" and x.shape[0] == H:
        R, sh, sr = x.shape[1], x.shape[1] * d, d
    elif layout == "batch" and x.shape[1] == H:
        R, sh, sr = x.shape[0], d, H * d
    else:
        raise AsmError("asm_whiten", ASM_ERR_INVALID_ARG)
    _check("asm_whiten", _lib.load().asm_whiten(
        _p(x), H, R, d, _dt(x), sh, sr, _p(mu), _p(W), _p(y), sh, sr, _stream(stream)))


def asm_decode_step_noalloc(q, centroids, a_bar, logz_bar, k_cache, v_cache, local_len,
                            scale: float, out, lse_out=None, idx_out=None, metric: int = ASM_L2,
                            flags: int = 0, stream=None):
    """asm_decode_step using the library's built-in scratch (no workspace argument)."""
    _contig(q, centroids, a_bar, logz_bar, k_cache, v_cache, local_len, out, lse_out, idx_out)
    B, Hq, d = q.shape
    K = centroids.shape[1]
    _, Hkv, Tmax, _ = k_cache.shape
    _check("asm_decode_step_noalloc", _lib.load().asm_decode_step_noalloc(
        _p(q), _p(centroids), _p(a_bar), _p(logz_bar), _p(k_cache), _p(v_cache), _p(local_len),
        B, Hq, Hkv, K, Tmax, d, float(scale), int(metric), _dt(q), _p(out), _p(lse_out),
        _p(idx_out), int(flags), _stream(stream)))


def asm_decode_noalloc_error(stream=None) -> int:
    """Device-side status of the last asm_decode_step_noalloc call on the current device."""
    code = ctypes.c_int(0)
    _check("asm_decode_noalloc_error", _lib.load().asm_decode_noalloc_error(ctypes.byref(code), _stream(stream)))
    return code.value


def asm_flash_decode(q, k_prefix, v_prefix, k_cache, v_cache, local_len, scale: float, out, ws,
                     lse_out=None, stream=None):
    """Full attention over a shared explicit prefix plus each row's local tokens."""
    _contig(q, k_prefix, v_prefix, k_cache, v_cache, local_len, out, lse_out)
    B, Hq, d = q.shape
    Hkv, Lp, _ = k_prefix.shape
    Tmax = k_cache.shape[2]
    _check("asm_flash_decode", _lib.load().asm_flash_decode(
        _p(q), _p(k_prefix), _p(v_prefix), Lp, _p(k_cache), _p(v_cache), _p(local_len), B, Hq, Hkv,
        Tmax, d, float(scale), _dt(q), _p(out), _p(lse_out), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


# ----------------------------------------------------------- paged serving --

def _want(fn: str, ok: bool) -> None:
    if not ok:
        raise AsmError(fn, ASM_ERR_INVALID_ARG)


def _take(fn: str, want: tuple, more: tuple = ()) -> int:
    """Every tensor on the current CUDA device, those of `want` contiguous;
    returns the device.  One short pass: a decode step makes several of these
    calls, and their host time is what a small one costs."""
    dev = want[0].get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse(fn, want[0], -1)
    for t in want:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            _refuse(fn, t, dev)
    for t in more:
        if t.get_device() != dev:
            _refuse(fn, t, dev)
    return dev


def _refuse(fn: str, t, dev: int) -> None:
    if t.device.type != "cuda":
        raise ValueError(f"{fn}: tensors must be on a CUDA device, got {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: tensors must all be on the current device, got {t.device}")
    raise ValueError(f"{fn}: tensors must be contiguous")


def _i32(fn: str, *ts) -> None:
    for t in ts:
        if t is not None and t.dtype is not torch.int32:
            raise TypeError(f"{fn}: lengths, ids and positions must be int32, got {t.dtype}")


def _f64(fn: str, t) -> None:
    if t.dtype is not torch.float64:
        raise TypeError(f"{fn}: freq must be float64, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(dev: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _heads(fn: str, t, T: int, d: int, dtype) -> tuple[int, int]:
    """Token and head strides of a [T, H, d] view whose heads are contiguous."""
    st = t.stride()
    if len(st) != 3 or t.shape[0] != T or t.shape[2] != d or t.dtype is not dtype:
        raise AsmError(fn, ASM_ERR_INVALID_ARG)
    if st[2] != 1:
        raise ValueError(f"{fn}: heads must be contiguous")
    return st[0], st[1]


def asm_page_step(kv_len, new_len, pool, pool_state, page_size: int, table, seq_len, q_off, row, pos, slot, pool_out,
                  pos_base=None, stream=None):
    """Page tables and slot maps of one step, from kv_len[R] and new_len[R]
    (negative: the row ends).  table[R,max_pages] and the ring pool[F] are
    updated; seq_len[R], q_off[R+1], row/pos/slot[T] and pool_out[3] written."""
    fn = "asm_page_step"
    dev = _take(fn, (kv_len, new_len, pos_base, pool, pool_state, table, seq_len, q_off, row, pos, slot, pool_out))
    _i32(fn, kv_len, new_len, pos_base, pool, pool_state, table, seq_len, q_off, row, pos, slot, pool_out)
    R, T = kv_len.numel(), row.numel()
    _want(fn, table.dim() == 2 and table.shape[0] == R and new_len.numel() == R and seq_len.numel() == R and
          q_off.numel() == R + 1 and pos.numel() == T and slot.numel() == T and pool_state.numel() == 3 and
          pool_out.numel() == 3 and (pos_base is None or pos_base.numel() == R))
    _check(fn, _lib.load().asm_page_step(
        kv_len.data_ptr(), new_len.data_ptr(), _ptr(pos_base), R, int(page_size), table.shape[1], table.data_ptr(),
        pool.data_ptr(), pool_state.data_ptr(), pool.numel(), T, seq_len.data_ptr(), q_off.data_ptr(), row.data_ptr(),
        pos.data_ptr(), slot.data_ptr(), pool_out.data_ptr(), _raw_stream(dev, stream)))


def asm_rope_freqs(freq, theta: float, scaling: int = ASM_ROPE_SCALE_NONE, factor: float = 1.0, lo: float = 1.0,
                   hi: float = 4.0, ctx: float = 8192.0, stream=None):
    """Angle per position of each rotated pair into freq[rot/2] (fp64)."""
    fn = "asm_rope_freqs"
    dev = _take(fn, (freq,))
    _f64(fn, freq)
    _check(fn, _lib.load().asm_rope_freqs(
        freq.data_ptr(), 2 * freq.numel(), float(theta), int(scaling), float(factor), float(lo), float(hi), float(ctx),
        _raw_stream(dev, stream)))


def asm_rope(x, pos, freq, y, layout: int = ASM_ROPE_HALF, mscale: float = 1.0, inverse: bool = False, stream=None):
    """Rotary positions of x[T,H,d] (any token and head strides) into y, which
    may be x; the first 2 * len(freq) elements of each head turn.  inverse
    turns back: the gradient of the call without it."""
    fn = "asm_rope"
    dev = _take(fn, (pos, freq), (x, y))
    _i32(fn, pos)
    _f64(fn, freq)
    T, H, d = x.shape
    _want(fn, y.shape == x.shape and pos.numel() == T)
    xs, ys = _heads(fn, x, T, d, x.dtype), _heads(fn, y, T, d, x.dtype)
    _check(fn, _lib.load().asm_rope(
        x.data_ptr(), *xs, T, H, d, _dt(x), pos.data_ptr(), freq.data_ptr(), 2 * freq.numel(), int(layout),
        float(mscale), 1 if inverse else 0, y.data_ptr(), *ys, _raw_stream(dev, stream)))


def asm_rope_append(q, k, v, pos, slot, freq, q_out, k_pages, v_pages, layout: int = ASM_ROPE_HALF,
                    mscale: float = 1.0, stream=None):
    """Rotary positions of q[T,Hq,d] into q_out (may be q) and of k[T,Hkv,d],
    which goes with v to the tokens' slots of k_pages, v_pages
    [n_pages,Hkv,S,d]; slots outside the pages store nothing."""
    fn = "asm_rope_append"
    dev = _take(fn, (pos, slot, freq, k_pages, v_pages), (q, k, v, q_out))
    _i32(fn, pos, slot)
    _f64(fn, freq)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    pages = k_pages.shape
    _want(fn, q_out.shape == q.shape and v.shape == k.shape and pos.numel() == T and slot.numel() == T and
          len(pages) == 4 and pages == v_pages.shape and pages[1] == Hkv and pages[3] == d and
          k_pages.dtype is q.dtype and v_pages.dtype is q.dtype)
    dt = q.dtype
    qs, ks, vs, os = _heads(fn, q, T, d, dt), _heads(fn, k, T, d, dt), _heads(fn, v, T, d, dt), _heads(fn, q_out, T, d, dt)
    _check(fn, _lib.load().asm_rope_append(
        q.data_ptr(), *qs, k.data_ptr(), *ks, v.data_ptr(), *vs, T, Hq, Hkv, d, _dt(q), pos.data_ptr(), slot.data_ptr(),
        freq.data_ptr(), 2 * freq.numel(), int(layout), float(mscale), q_out.data_ptr(), *os, k_pages.data_ptr(),
        v_pages.data_ptr(), pages[0], pages[2], _raw_stream(dev, stream)))


def asm_shared_plan_size(R: int, NG: int, T: int, Hq: int, Hkv: int) -> int:
    return int(_lib.load().asm_shared_plan_size(R, NG, T, Hq, Hkv))


def asm_shared_plan(q_off, seq_len, table, T: int, Hq: int, Hkv: int, page_size: int, plan, group_off=None,
                    prefix_len=None, prefix_table=None, stream=None):
    """The work list of asm_shared_attention for a step's lengths: q_off[R+1],
    seq_len[R], and the rows group_off[NG+1] that share each prefix of
    prefix_len[NG] tokens (the tables give the page limits only)."""
    fn = "asm_shared_plan"
    dev = _take(fn, (q_off, seq_len, table, group_off, prefix_len, prefix_table, plan))
    _i32(fn, q_off, seq_len, table, group_off, prefix_len, prefix_table)
    R = seq_len.numel()
    NG = 0 if group_off is None else group_off.numel() - 1
    _want(fn, table.dim() == 2 and table.shape[0] == R and q_off.numel() == R + 1)
    _want(fn, NG <= 0 or (prefix_len is not None and prefix_table is not None and prefix_len.numel() == NG and
                          prefix_table.dim() == 2 and prefix_table.shape[0] == NG))
    _check(fn, _lib.load().asm_shared_plan(
        q_off.data_ptr(), seq_len.data_ptr(), _ptr(group_off), _ptr(prefix_len), R, NG, int(T), int(Hq),
        int(Hkv), int(page_size), table.shape[1], prefix_table.shape[1] if NG > 0 else 0, plan.data_ptr(), plan.numel() * plan.element_size(),
        _raw_stream(dev, stream)))


def asm_shared_attention_workspace_size(T: int, Hq: int, Hkv: int, d: int) -> int:
    return int(_lib.load().asm_shared_attention_workspace_size(T, Hq, Hkv, d))


def asm_shared_attention(q, k_pages, v_pages, table, plan, scale: float, out, ws, prefix_table=None, lse_out=None,
                         stream=None):
    """Attention of the tokens q[T,Hq,d] over their rows' shared prefixes and
    local pages [n_pages,Hkv,S,d] into out[T,Hq,d] (and lse_out[T,Hq])."""
    fn = "asm_shared_attention"
    dev = _take(fn, (q, k_pages, v_pages, table, plan, out, ws, prefix_table, lse_out))
    _i32(fn, table, prefix_table)
    T, Hq, d = q.shape
    pages, dt = k_pages.shape, q.dtype
    NG = 0 if prefix_table is None else prefix_table.shape[0]
    _want(fn, len(pages) == 4 and pages == v_pages.shape and pages[3] == d and out.shape == q.shape and
          table.dim() == 2 and (prefix_table is None or prefix_table.dim() == 2) and out.dtype is dt and
          k_pages.dtype is dt and v_pages.dtype is dt)
    _want(fn, lse_out is None or (lse_out.dtype is torch.float32 and lse_out.numel() == T * Hq))
    _check(fn, _lib.load().asm_shared_attention(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), pages[0], pages[2], table.data_ptr(), table.shape[1],
        _ptr(prefix_table), prefix_table.shape[1] if NG else 0, plan.data_ptr(), plan.numel() * plan.element_size(),
        table.shape[0], NG, T, Hq, pages[1], d, float(scale), _dt(q), out.data_ptr(), _ptr(lse_out), ws.data_ptr(),
        ws.numel() * ws.element_size(), _raw_stream(dev, stream)))


# ---------------------------------------------------------------- helpers --

def asm_index_reorder(perm, centroids, a_bar, logz_bar, centroids_ord, a_bar_ord, logz_bar_ord, stream=None):
    """Lay a memory out by cluster: row i of head h <- row perm[h, i]."""
    _contig(perm, centroids, a_bar, logz_bar, centroids_ord, a_bar_ord, logz_bar_ord)
    H, K, d = centroids.shape
    _check("asm_index_reorder", _lib.load().asm_index_reorder(
        _p(perm), H, K, d, _dt(centroids), _p(centroids), _p(a_bar), _p(logz_bar), _p(centroids_ord),
        _p(a_bar_ord), _p(logz_bar_ord), _stream(stream)))


def asm_decode_indexed_workspace_size(B, Hq, Hkv, K1, P, max_seg, Tmax, d, dtype) -> int:
    return int(_lib.load().asm_decode_indexed_workspace_size(B, Hq, Hkv, K1, P, max_seg, Tmax, d, _DT[dtype]))


def asm_decode_step_indexed(q, supers, seg_off, P: int, max_seg: int, centroids, a_bar, logz_bar, k_cache,
                            v_cache, local_len, scale: float, out, ws, lse_out=None, idx_out=None,
                            metric: int = ASM_L2, stream=None):
    """Decode step with the two-level search over a memory ordered by cluster."""
    _contig(q, supers, seg_off, centroids, a_bar, logz_bar, k_cache, v_cache, local_len, out, lse_out, idx_out)
    B, Hq, d = q.shape
    K1 = supers.shape[1]
    K = centroids.shape[1]
    Hkv, Tmax = k_cache.shape[1], k_cache.shape[2]
    _check("asm_decode_step_indexed", _lib.load().asm_decode_step_indexed(
        _p(q), _p(supers), _p(seg_off), K1, int(P), int(max_seg), _p(centroids), _p(a_bar), _p(logz_bar),
        _p(k_cache), _p(v_cache), _p(local_len), B, Hq, Hkv, K, Tmax, d, float(scale), int(metric), _dt(q),
        _p(out), _p(lse_out), _p(idx_out), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def alloc_workspace(nbytes: int, device, zero: bool = True) -> torch.Tensor:
    """A 256-byte-granular device buffer (zeroed: ready for decode calls)."""
    n = max(256, (int(nbytes) + 255) // 256 * 256)
    t = torch.empty(n, dtype=torch.uint8, device=device)
    if zero:
        asm_workspace_init(t)
    return t
