"""Lossless draft verification with self-selection on MI355X (gfx950).

Thin ctypes binding over ``libsvd.so`` (C ABI in ``include/svd.h``).  Every step
of the verification runs in the library's HIP kernels; this module only
marshals arguments.  PyTorch supplies device memory and the current stream.

Raw entry points (same names and argument order as the C ABI; pointer
arguments take an int address or a tensor):
    svd_workspace_bytes, svd_verify, svd_select_and_verify, svd_greedy_verify,
    svd_greedy_select_and_verify, svd_rows_workspace_bytes, svd_select_and_verify_rows,
    svd_verify_window, svd_cps_workspace_bytes, svd_cps_lattice, svd_cps_beam,
    svd_adl_next, svd_select_and_verify_noalloc, svd_strerror; around the verification step:
    svd_draft_tree, svd_cache_write, svd_cache_read, svd_tree_attention_workspace_bytes,
    svd_tree_attention, svd_adjust_logits, svd_cache_pages_workspace_bytes, svd_cache_pages,
    svd_cache_slots, svd_cache_write_slots, svd_filter_logits, svd_sample,
    svd_prefix_attention_workspace_bytes, svd_prefix_attention
Tensor conveniences that allocate the outputs and the workspace with torch:
    verify, select_and_verify, greedy_verify, greedy_select_and_verify,
    select_and_verify_rows, verify_window, cps_lattice, cps_beam, adl_next, workspace_bytes;
    draft_tree, kv_cache, cache_write, cache_read, tree_attention, adjust_logits;
    page_pool, cache_pages, cache_slots, cache_write_slots, filter_logits, sample,
    prefix_attention
  Their stream argument is the handle of the stream to run on (an int; default the
  current one); what a call allocates, its results too, belongs to that stream.
Kernel timing: timing_library() loads ``libsvd_timed.so`` (the same kernels with
HIP-event timing compiled in, ``include/svd_timing.h``) as a Library whose raw
entry points are those above plus svd_profile_enable and svd_profile_read.

Importing fails with ImportError when ``libsvd.so`` has not been built; there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvd.so")
TIMED_LIB_PATH = os.path.join(_PKG, "libsvd_timed.so")

SVD_F32, SVD_BF16 = 0, 1
SVD_OK, SVD_EINVAL, SVD_EDTYPE, SVD_EWORKSPACE, SVD_EHIP, SVD_ESCRATCH = 0, -1, -2, -3, -4, -5
SVD_NOALLOC_SCRATCH_BYTES = 16 << 20
SVD_MAX_K, SVD_MAX_GAMMA = 64, 4096
SVD_MAX_NODES = 4096
SVD_CACHE_BF16, SVD_CACHE_E4M3 = 0, 1
# kernel ids of the timing build (SVD_KERNEL_* in include/svd_timing.h)
KERNELS = ("rowstats", "select", "draw_pass", "draw_pick", "beta", "mark", "pool_stats",
           "alpha_rows", "lattice", "beam", "lattice_len", "combine", "rowstats_split",
           "rowstats_live", "adl", "beta_combine", "draft_tree", "cache_write", "cache_read",
           "tree_attention", "attention_join", "adjust", "pages", "slots", "filter", "sample", "share",
           "shared_attention")
SVD_RULE_STANDARD, SVD_RULE_GREEDY = 0, 1

C_EXPORTS = ("svd_workspace_bytes", "svd_verify", "svd_select_and_verify", "svd_greedy_verify",
             "svd_greedy_select_and_verify", "svd_rows_workspace_bytes",
             "svd_select_and_verify_rows", "svd_verify_window", "svd_cps_workspace_bytes",
             "svd_cps_lattice", "svd_cps_beam", "svd_adl_next", "svd_select_and_verify_noalloc",
             "svd_draft_tree", "svd_cache_write", "svd_cache_read",
             "svd_tree_attention_workspace_bytes", "svd_tree_attention", "svd_adjust_logits",
             "svd_cache_pages_workspace_bytes", "svd_cache_pages", "svd_cache_slots",
             "svd_cache_write_slots", "svd_filter_logits", "svd_sample",
             "svd_prefix_attention_workspace_bytes", "svd_prefix_attention", "svd_strerror")
TIMING_EXPORTS = ("svd_profile_enable", "svd_profile_read")

_M64 = 0xFFFFFFFFFFFFFFFF


class CacheStruct(ctypes.Structure):
    """svd_cache_t of include/svd.h; pointers are int addresses."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("page", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class SvdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, svd_strerror(status), status))


def _declare(L: ctypes.CDLL, timing: bool) -> ctypes.CDLL:
    vp, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.c_uint64, ctypes.c_float, ctypes.c_size_t)
    L.svd_workspace_bytes.restype = sz
    L.svd_workspace_bytes.argtypes = [i64, i32, i32, i32]
    L.svd_verify.restype = ctypes.c_int
    L.svd_verify.argtypes = [vp, vp, vp, ctypes.c_int, i64, i32, i32, f32, f32, u64, u64,
                             vp, vp, vp, vp, vp, sz, vp]
    L.svd_select_and_verify.restype = ctypes.c_int
    L.svd_select_and_verify.argtypes = [vp, vp, vp, ctypes.c_int, i64, i32, i32, i32, f32, f32,
                                        u64, u64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.svd_greedy_verify.restype = ctypes.c_int
    L.svd_greedy_verify.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, f32, u64, u64, vp, vp,
                                    vp, vp, sz, vp]
    L.svd_greedy_select_and_verify.restype = ctypes.c_int
    L.svd_greedy_select_and_verify.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, i32, f32, u64,
                                               u64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.svd_rows_workspace_bytes.restype = sz
    L.svd_rows_workspace_bytes.argtypes = [i64, i32, i32, i32, i64, i64]
    L.svd_select_and_verify_rows.restype = ctypes.c_int
    L.svd_select_and_verify_rows.argtypes = [ctypes.c_int, vp, i64, vp, vp, i64, vp, vp,
                                             ctypes.c_int, i64, i32, i32, i32, f32, f32, u64, u64,
                                             vp, vp, vp, vp, vp, vp, sz, vp]
    L.svd_verify_window.restype = ctypes.c_int
    L.svd_verify_window.argtypes = [ctypes.c_int, vp, vp, vp, vp, i32, i32, ctypes.c_int, i64, i32,
                                    i32, i32, f32, f32, u64, u64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.svd_cps_workspace_bytes.restype = sz
    L.svd_cps_workspace_bytes.argtypes = [i64, i32]
    L.svd_cps_lattice.restype = ctypes.c_int
    L.svd_cps_lattice.argtypes = [vp, ctypes.c_int, i64, i32, i32, f32, f32, i32, i32, vp, vp, vp,
                                  vp, vp, sz, vp]
    L.svd_cps_beam.restype = ctypes.c_int
    L.svd_cps_beam.argtypes = [vp, vp, vp, vp, vp, f32, i64, i32, i32, i32, vp, vp, vp, vp]
    L.svd_adl_next.restype = ctypes.c_int
    L.svd_adl_next.argtypes = [vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32, i32, i32, vp, vp,
                               vp]
    L.svd_select_and_verify_noalloc.restype = ctypes.c_int
    L.svd_select_and_verify_noalloc.argtypes = [vp, vp, vp, ctypes.c_int, i64, i32, i32, i32, f32,
                                                f32, u64, u64, vp, vp, vp, vp, vp, vp, vp]
    L.svd_draft_tree.restype = ctypes.c_int
    L.svd_draft_tree.argtypes = [vp, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.svd_cache_write.restype = ctypes.c_int
    L.svd_cache_write.argtypes = [vp, vp, vp, ctypes.c_int, i64, i64, vp, vp, vp, i64, i64, vp]
    L.svd_cache_read.restype = ctypes.c_int
    L.svd_cache_read.argtypes = [vp, vp, vp, i64, i64, ctypes.c_int, vp, vp, vp]
    L.svd_tree_attention_workspace_bytes.restype = sz
    L.svd_tree_attention_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i64]
    L.svd_tree_attention.restype = ctypes.c_int
    L.svd_tree_attention.argtypes = [vp, vp, i64, vp, vp, vp, f32, i64, i32, i32, vp, vp, vp, sz,
                                     vp]
    L.svd_adjust_logits.restype = ctypes.c_int
    L.svd_adjust_logits.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, vp, vp, i64, vp, vp, vp,
                                    vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, i32, vp]
    L.svd_cache_pages_workspace_bytes.restype = sz
    L.svd_cache_pages_workspace_bytes.argtypes = [i64]
    L.svd_cache_pages.restype = ctypes.c_int
    L.svd_cache_pages.argtypes = [vp, vp, i64, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  sz, vp]
    L.svd_cache_slots.restype = ctypes.c_int
    L.svd_cache_slots.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, vp, vp, vp, vp, vp]
    L.svd_cache_write_slots.restype = ctypes.c_int
    L.svd_cache_write_slots.argtypes = [vp, vp, vp, ctypes.c_int, i64, i64, vp, i64, vp]
    L.svd_filter_logits.restype = ctypes.c_int
    L.svd_filter_logits.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, vp, vp, vp, vp, vp, vp]
    L.svd_sample.restype = ctypes.c_int
    L.svd_sample.argtypes = [vp, ctypes.c_int, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, u64, u64,
                             vp, vp, vp]
    L.svd_prefix_attention_workspace_bytes.restype = sz
    L.svd_prefix_attention_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i64, i64]
    L.svd_prefix_attention.restype = ctypes.c_int
    L.svd_prefix_attention.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, i64, f32, f32, vp, i64, i32,
                                       i32, vp, vp, vp, sz, vp]
    L.svd_strerror.restype = ctypes.c_char_p
    L.svd_strerror.argtypes = [ctypes.c_int]
    if timing:
        L.svd_profile_enable.restype = ctypes.c_int
        L.svd_profile_enable.argtypes = [ctypes.c_uint]
        L.svd_profile_read.restype = ctypes.c_int
        L.svd_profile_read.argtypes = [vp, vp, ctypes.c_int]
    return L


def _addr(x):
    """Device address of a tensor, an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _struct(c):
    """Address of a CacheStruct, or None."""
    return None if c is None else ctypes.addressof(c)


class Library:
    """The raw C ABI of one built library (argument marshalling only)."""

    def __init__(self, path: str = LIB_PATH, timing: bool = False):
        if not os.path.exists(path):
            raise ImportError(
                "%s is not built (expected at %s); build it with __graft_entry__.build() or "
                "python -m lossless_draft_verification_verifier_amd._build"
                % (os.path.basename(path), path))
        self.path = path
        self.timing = timing
        self._lib = _declare(ctypes.CDLL(path), timing)

    def svd_workspace_bytes(self, B: int, K: int, gamma: int, V: int) -> int:
        return int(self._lib.svd_workspace_bytes(B, K, gamma, V))

    def svd_verify(self, p_logits, q_logits, draft, dtype, B, gamma, V, temp_p, temp_q, seed,
                   row_base, accept_len, next_token, alpha, beta, workspace, workspace_bytes,
                   hip_stream) -> int:
        return int(self._lib.svd_verify(
            _addr(p_logits), _addr(q_logits), _addr(draft), int(dtype), int(B), int(gamma),
            int(V), float(temp_p), float(temp_q), int(seed) & _M64, int(row_base) & _M64,
            _addr(accept_len), _addr(next_token), _addr(alpha), _addr(beta), _addr(workspace),
            int(workspace_bytes), _addr(hip_stream)))

    def svd_select_and_verify(self, p_logits, q_logits, drafts, dtype, B, K, gamma, V, temp_p,
                              temp_q, seed, row_base, selected, accept_len, next_token, scores,
                              alpha, beta, workspace, workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_select_and_verify(
            _addr(p_logits), _addr(q_logits), _addr(drafts), int(dtype), int(B), int(K),
            int(gamma), int(V), float(temp_p), float(temp_q), int(seed) & _M64,
            int(row_base) & _M64, _addr(selected), _addr(accept_len), _addr(next_token),
            _addr(scores), _addr(alpha), _addr(beta), _addr(workspace), int(workspace_bytes),
            _addr(hip_stream)))

    def svd_greedy_verify(self, p_logits, draft, dtype, B, gamma, V, temp_p, seed, row_base,
                          accept_len, next_token, alpha, workspace, workspace_bytes,
                          hip_stream) -> int:
        return int(self._lib.svd_greedy_verify(
            _addr(p_logits), _addr(draft), int(dtype), int(B), int(gamma), int(V), float(temp_p),
            int(seed) & _M64, int(row_base) & _M64, _addr(accept_len), _addr(next_token),
            _addr(alpha), _addr(workspace), int(workspace_bytes), _addr(hip_stream)))

    def svd_greedy_select_and_verify(self, p_logits, drafts, dtype, B, K, gamma, V, temp_p, seed,
                                     row_base, selected, accept_len, next_token, scores, alpha,
                                     workspace, workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_greedy_select_and_verify(
            _addr(p_logits), _addr(drafts), int(dtype), int(B), int(K), int(gamma), int(V),
            float(temp_p), int(seed) & _M64, int(row_base) & _M64, _addr(selected),
            _addr(accept_len), _addr(next_token), _addr(scores), _addr(alpha), _addr(workspace),
            int(workspace_bytes), _addr(hip_stream)))

    def svd_rows_workspace_bytes(self, B: int, K: int, gamma: int, V: int, n_p_rows: int,
                                 n_q_rows: int) -> int:
        return int(self._lib.svd_rows_workspace_bytes(B, K, gamma, V, n_p_rows, n_q_rows))

    def svd_select_and_verify_rows(self, rule, p_rows, n_p_rows, p_index, q_rows, n_q_rows,
                                   q_index, drafts, dtype, B, K, gamma, V, temp_p, temp_q, seed,
                                   row_base, selected, accept_len, next_token, scores, alpha,
                                   workspace, workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_select_and_verify_rows(
            int(rule), _addr(p_rows), int(n_p_rows), _addr(p_index), _addr(q_rows),
            int(n_q_rows), _addr(q_index), _addr(drafts), int(dtype), int(B), int(K), int(gamma),
            int(V), float(temp_p), float(temp_q), int(seed) & _M64, int(row_base) & _M64,
            _addr(selected), _addr(accept_len), _addr(next_token), _addr(scores), _addr(alpha),
            _addr(workspace), int(workspace_bytes), _addr(hip_stream)))

    def svd_verify_window(self, rule, p_logits, q_logits, drafts, gamma_b, eos, early_exit, dtype,
                          B, K, gamma, V, temp_p, temp_q, seed, row_base, selected, accept_len,
                          next_token, scores, alpha, workspace, workspace_bytes,
                          hip_stream) -> int:
        return int(self._lib.svd_verify_window(
            int(rule), _addr(p_logits), _addr(q_logits), _addr(drafts), _addr(gamma_b), int(eos),
            int(early_exit), int(dtype), int(B), int(K), int(gamma), int(V), float(temp_p),
            float(temp_q), int(seed) & _M64, int(row_base) & _M64, _addr(selected),
            _addr(accept_len), _addr(next_token), _addr(scores), _addr(alpha), _addr(workspace),
            int(workspace_bytes), _addr(hip_stream)))

    def svd_cps_workspace_bytes(self, B: int, G: int) -> int:
        return int(self._lib.svd_cps_workspace_bytes(B, G))

    def svd_cps_lattice(self, q_logits, dtype, B, G, V, temp_q, tau, m_max, eos, cand, cand_logp,
                        n_cand, length, workspace, workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_cps_lattice(
            _addr(q_logits), int(dtype), int(B), int(G), int(V), float(temp_q), float(tau),
            int(m_max), int(eos), _addr(cand), _addr(cand_logp), _addr(n_cand), _addr(length),
            _addr(workspace), int(workspace_bytes), _addr(hip_stream)))

    def svd_cps_beam(self, cand, cand_logp, n_cand, length, fluency, lam, B, G, m_max, beam,
                     paths, path_score, path_len, hip_stream) -> int:
        return int(self._lib.svd_cps_beam(
            _addr(cand), _addr(cand_logp), _addr(n_cand), _addr(length), _addr(fluency),
            float(lam), int(B), int(G), int(m_max), int(beam), _addr(paths), _addr(path_score),
            _addr(path_len), _addr(hip_stream)))

    def svd_adl_next(self, drafts, selected, accept_len, gamma_b, eos, B, K, gamma, k_min, k_max,
                     step, shift, slack, avg, next_gamma, hip_stream) -> int:
        return int(self._lib.svd_adl_next(
            _addr(drafts), _addr(selected), _addr(accept_len), _addr(gamma_b), int(eos), int(B),
            int(K), int(gamma), int(k_min), int(k_max), int(step), int(shift), int(slack),
            _addr(avg), _addr(next_gamma), _addr(hip_stream)))

    def svd_select_and_verify_noalloc(self, p_logits, q_logits, drafts, dtype, B, K, gamma, V,
                                      temp_p, temp_q, seed, row_base, selected, accept_len,
                                      next_token, scores, alpha, beta, hip_stream) -> int:
        return int(self._lib.svd_select_and_verify_noalloc(
            _addr(p_logits), _addr(q_logits), _addr(drafts), int(dtype), int(B), int(K),
            int(gamma), int(V), float(temp_p), float(temp_q), int(seed) & _M64,
            int(row_base) & _M64, _addr(selected), _addr(accept_len), _addr(next_token),
            _addr(scores), _addr(alpha), _addr(beta), _addr(hip_stream)))

    def svd_draft_tree(self, drafts, root, B, K, gamma, T, tokens, parent, depth, anc, n_nodes,
                       p_index, hip_stream) -> int:
        return int(self._lib.svd_draft_tree(
            _addr(drafts), _addr(root), int(B), int(K), int(gamma), int(T), _addr(tokens),
            _addr(parent), _addr(depth), _addr(anc), _addr(n_nodes), _addr(p_index),
            _addr(hip_stream)))

    def svd_cache_write(self, cache, k, v, dtype, k_stride, v_stride, ctx_len, n_new, dst, B, T,
                        hip_stream) -> int:
        return int(self._lib.svd_cache_write(
            _struct(cache), _addr(k), _addr(v), int(dtype), int(k_stride), int(v_stride),
            _addr(ctx_len), _addr(n_new), _addr(dst), int(B), int(T), _addr(hip_stream)))

    def svd_cache_read(self, cache, start, count, B, N, dtype, k, v, hip_stream) -> int:
        return int(self._lib.svd_cache_read(
            _struct(cache), _addr(start), _addr(count), int(B), int(N), int(dtype), _addr(k),
            _addr(v), _addr(hip_stream)))

    def svd_tree_attention_workspace_bytes(self, B: int, T: int, q_heads: int, kv_heads: int,
                                           head_dim: int, max_len: int) -> int:
        return int(self._lib.svd_tree_attention_workspace_bytes(B, T, q_heads, kv_heads, head_dim,
                                                                max_len))

    def svd_tree_attention(self, cache, q, q_stride, ctx_len, n_nodes, anc, scale, B, T, q_heads,
                           out, lse, workspace, workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_tree_attention(
            _struct(cache), _addr(q), int(q_stride), _addr(ctx_len), _addr(n_nodes), _addr(anc),
            float(scale), int(B), int(T), int(q_heads), _addr(out), _addr(lse), _addr(workspace),
            int(workspace_bytes), _addr(hip_stream)))

    def svd_adjust_logits(self, logits, out, dtype, B, T, V, n_rows, history, hist_stride,
                          hist_len, prompt_len, tokens, anc, repetition, frequency, presence,
                          bias_off, bias_tok, bias_val, n_bias, allow, allow_index, n_masks,
                          hip_stream) -> int:
        return int(self._lib.svd_adjust_logits(
            _addr(logits), _addr(out), int(dtype), int(B), int(T), int(V), _addr(n_rows),
            _addr(history), int(hist_stride), _addr(hist_len), _addr(prompt_len), _addr(tokens),
            _addr(anc), _addr(repetition), _addr(frequency), _addr(presence), _addr(bias_off),
            _addr(bias_tok), _addr(bias_val), int(n_bias), _addr(allow), _addr(allow_index),
            int(n_masks), _addr(hip_stream)))

    def svd_cache_pages_workspace_bytes(self, B: int) -> int:
        return int(self._lib.svd_cache_pages_workspace_bytes(B))

    def svd_cache_pages(self, length, shared, B, max_pages, page, n_pages, free_ring, state, held,
                        block_table, state_out, held_out, table_out, room, workspace,
                        workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_cache_pages(
            _addr(length), _addr(shared), int(B), int(max_pages), int(page), int(n_pages),
            _addr(free_ring), _addr(state), _addr(held), _addr(block_table), _addr(state_out),
            _addr(held_out), _addr(table_out), _addr(room), _addr(workspace),
            int(workspace_bytes), _addr(hip_stream)))

    def svd_cache_slots(self, ctx_len, n_new, block_table, B, max_pages, page, n_pages, N, row_off,
                        seq, pos, slot, hip_stream) -> int:
        return int(self._lib.svd_cache_slots(
            _addr(ctx_len), _addr(n_new), _addr(block_table), int(B), int(max_pages), int(page),
            int(n_pages), int(N), _addr(row_off), _addr(seq), _addr(pos), _addr(slot),
            _addr(hip_stream)))

    def svd_cache_write_slots(self, cache, k, v, dtype, k_stride, v_stride, slot, N,
                              hip_stream) -> int:
        return int(self._lib.svd_cache_write_slots(
            _struct(cache), _addr(k), _addr(v), int(dtype), int(k_stride), int(v_stride),
            _addr(slot), int(N), _addr(hip_stream)))

    def svd_filter_logits(self, logits, out, dtype, B, T, V, n_rows, temperature, top_k, top_p,
                          min_p, hip_stream) -> int:
        return int(self._lib.svd_filter_logits(
            _addr(logits), _addr(out), int(dtype), int(B), int(T), int(V), _addr(n_rows),
            _addr(temperature), _addr(top_k), _addr(top_p), _addr(min_p), _addr(hip_stream)))

    def svd_sample(self, logits, dtype, B, T, V, K, n_rows, temperature, top_k, top_p, min_p,
                   uniforms, seed, row_base, token, logprob, hip_stream) -> int:
        return int(self._lib.svd_sample(
            _addr(logits), int(dtype), int(B), int(T), int(V), int(K), _addr(n_rows),
            _addr(temperature), _addr(top_k), _addr(top_p), _addr(min_p), _addr(uniforms),
            int(seed) & _M64, int(row_base) & _M64, _addr(token), _addr(logprob),
            _addr(hip_stream)))

    def svd_prefix_attention_workspace_bytes(self, B: int, T: int, q_heads: int, kv_heads: int,
                                             head_dim: int, max_len: int, n_groups: int) -> int:
        return int(self._lib.svd_prefix_attention_workspace_bytes(B, T, q_heads, kv_heads,
                                                                  head_dim, max_len, n_groups))

    def svd_prefix_attention(self, cache, q, q_stride, ctx_len, n_nodes, anc, depth, share_off,
                             n_groups, scale, cap, slopes, B, T, q_heads, out, lse, workspace,
                             workspace_bytes, hip_stream) -> int:
        return int(self._lib.svd_prefix_attention(
            _struct(cache), _addr(q), int(q_stride), _addr(ctx_len), _addr(n_nodes), _addr(anc),
            _addr(depth), _addr(share_off), int(n_groups), float(scale), float(cap),
            _addr(slopes), int(B), int(T), int(q_heads), _addr(out), _addr(lse), _addr(workspace),
            int(workspace_bytes), _addr(hip_stream)))

    def svd_strerror(self, status: int) -> str:
        return self._lib.svd_strerror(int(status)).decode()

    # -- the timing build only ------------------------------------------------
    def svd_profile_enable(self, kernels=()) -> int:
        """Time the named kernels (names from KERNELS; "all" for every one) in
        later calls; an empty selection stops timing."""
        if not self.timing:
            raise RuntimeError("kernel timing needs the timing build (timing_library())")
        if kernels == "all":
            kernels = KERNELS
        mask = 0
        for k in kernels:
            mask |= 1 << KERNELS.index(k)
        return int(self._lib.svd_profile_enable(mask))

    def svd_profile_read(self):
        """(milliseconds per kernel, launches per kernel), indexed like KERNELS."""
        if not self.timing:
            raise RuntimeError("kernel timing needs the timing build (timing_library())")
        n = len(KERNELS)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        st = self._lib.svd_profile_read(ctypes.cast(ms, ctypes.c_void_p),
                                        ctypes.cast(cnt, ctypes.c_void_p), n)
        if st != SVD_OK:
            raise SvdError(st, "svd_profile_read")
        return list(ms), list(cnt)


_default = Library(LIB_PATH)
_c = _default._lib
_timed = []


def timing_library() -> Library:
    """The timing build, loaded once (ImportError when it is not built)."""
    if not _timed:
        _timed.append(Library(TIMED_LIB_PATH, timing=True))
    return _timed[0]


svd_workspace_bytes = _default.svd_workspace_bytes
svd_verify = _default.svd_verify
svd_select_and_verify = _default.svd_select_and_verify
svd_greedy_verify = _default.svd_greedy_verify
svd_greedy_select_and_verify = _default.svd_greedy_select_and_verify
svd_rows_workspace_bytes = _default.svd_rows_workspace_bytes
svd_select_and_verify_rows = _default.svd_select_and_verify_rows
svd_verify_window = _default.svd_verify_window
svd_cps_workspace_bytes = _default.svd_cps_workspace_bytes
svd_cps_lattice = _default.svd_cps_lattice
svd_cps_beam = _default.svd_cps_beam
svd_select_and_verify_noalloc = _default.svd_select_and_verify_noalloc
svd_adl_next = _default.svd_adl_next
svd_draft_tree = _default.svd_draft_tree
svd_cache_write = _default.svd_cache_write
svd_cache_read = _default.svd_cache_read
svd_tree_attention_workspace_bytes = _default.svd_tree_attention_workspace_bytes
svd_tree_attention = _default.svd_tree_attention
svd_adjust_logits = _default.svd_adjust_logits
svd_cache_pages_workspace_bytes = _default.svd_cache_pages_workspace_bytes
svd_cache_pages = _default.svd_cache_pages
svd_cache_slots = _default.svd_cache_slots
svd_cache_write_slots = _default.svd_cache_write_slots
svd_filter_logits = _default.svd_filter_logits
svd_sample = _default.svd_sample
svd_prefix_attention_workspace_bytes = _default.svd_prefix_attention_workspace_bytes
svd_prefix_attention = _default.svd_prefix_attention
svd_strerror = _default.svd_strerror


# --------------------------------------------------------------------------
# Tensor conveniences

_T = None  # torch, once a convenience has been called


def _torch():
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


def _on(stream, t, f, *args):
    """f(*args) on `stream` (its handle, an int) of t's device.  What f allocates has to
    belong to that stream: memory of the current one may still be in use there, and goes
    back to it when its tensor is dropped, while the call still runs.  The results are
    marked as used on the current stream as well, which is where the caller drops them."""
    torch = _torch()
    dev = t.get_device()
    if dev < 0 or stream == torch._C._cuda_getCurrentRawStream(dev):
        return f(*args)
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
        r = f(*args)
    for x in r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else (r,):
        if x is not None:
            x.record_stream(here)
    return r


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return SVD_BF16
    if t.dtype == torch.float32:
        return SVD_F32
    raise TypeError("logits must be torch.bfloat16 or torch.float32, got %s" % t.dtype)


def _check(t, name, device):
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def workspace_bytes(B, K, gamma, V) -> int:
    n = svd_workspace_bytes(B, K, gamma, V)
    if n == 0:
        raise ValueError("sizes out of range: B=%d K=%d gamma=%d V=%d" % (B, K, gamma, V))
    return n


def alloc_workspace(B, K, gamma, V, device):
    import torch
    n = workspace_bytes(B, K, gamma, V)
    return torch.empty(n, dtype=torch.uint8, device=device)  # torch allocations are 256-B aligned


def select_and_verify(p, q, drafts, temp_p=1.0, temp_q=None, seed=0, row_base=0,
                      want_alpha=False, want_beta=False, want_scores=False, workspace=None,
                      stream=None):
    """p [B,K,gamma+1,V], q [B,K,gamma,V] (bf16 or fp32), drafts [B,K,gamma] int32."""
    if stream is not None:
        return _on(stream, p, select_and_verify, p, q, drafts, temp_p, temp_q, seed, row_base,
                   want_alpha, want_beta, want_scores, workspace)
    import torch
    dev = p.device
    for t, n in ((p, "p"), (q, "q"), (drafts, "drafts")):
        _check(t, n, dev)
    if drafts.dtype != torch.int32:
        raise TypeError("drafts must be int32")
    if p.dtype != q.dtype:
        raise TypeError("p and q must share one dtype")
    if p.dim() != 4 or q.dim() != 4 or drafts.dim() != 3:
        raise ValueError("expected p [B,K,G+1,V], q [B,K,G,V], drafts [B,K,G]")
    B, K, G1, V = p.shape
    G = G1 - 1
    if tuple(q.shape) != (B, K, G, V) or tuple(drafts.shape) != (B, K, G):
        raise ValueError("shape mismatch: p %s q %s drafts %s" % (tuple(p.shape), tuple(q.shape),
                                                                 tuple(drafts.shape)))
    temp_q = temp_p if temp_q is None else temp_q
    out = {
        "selected": torch.empty(B, dtype=torch.int32, device=dev),
        "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
        "next_token": torch.empty(B, dtype=torch.int32, device=dev),
        "scores": torch.empty((B, K), dtype=torch.float32, device=dev) if want_scores else None,
        "alpha": torch.empty((B, K, G), dtype=torch.float32, device=dev) if want_alpha else None,
        "beta": torch.empty((B, K, G), dtype=torch.float32, device=dev) if want_beta else None,
    }
    ws = alloc_workspace(B, K, G, V, dev) if workspace is None else workspace
    _check(ws, "workspace", dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    rc = svd_select_and_verify(p, q, drafts, _dtype_code(p), B, K, G, V, temp_p, temp_q, seed,
                               row_base, out["selected"], out["accept_len"], out["next_token"],
                               out["scores"], out["alpha"], out["beta"], ws, ws.numel(), st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_select_and_verify")
    return out


def verify(p, q, draft, temp_p=1.0, temp_q=None, seed=0, row_base=0, want_alpha=False,
           want_beta=False, workspace=None, stream=None):
    """p [B,gamma+1,V], q [B,gamma,V] (bf16 or fp32), draft [B,gamma] int32."""
    if stream is not None:
        return _on(stream, p, verify, p, q, draft, temp_p, temp_q, seed, row_base, want_alpha,
                   want_beta, workspace)
    import torch
    dev = p.device
    for t, n in ((p, "p"), (q, "q"), (draft, "draft")):
        _check(t, n, dev)
    if draft.dtype != torch.int32:
        raise TypeError("draft must be int32")
    if p.dtype != q.dtype:
        raise TypeError("p and q must share one dtype")
    B, G1, V = p.shape
    G = G1 - 1
    if tuple(q.shape) != (B, G, V) or tuple(draft.shape) != (B, G):
        raise ValueError("shape mismatch")
    temp_q = temp_p if temp_q is None else temp_q
    out = {
        "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
        "next_token": torch.empty(B, dtype=torch.int32, device=dev),
        "alpha": torch.empty((B, G), dtype=torch.float32, device=dev) if want_alpha else None,
        "beta": torch.empty((B, G), dtype=torch.float32, device=dev) if want_beta else None,
    }
    ws = alloc_workspace(B, 1, G, V, dev) if workspace is None else workspace
    _check(ws, "workspace", dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    rc = svd_verify(p, q, draft, _dtype_code(p), B, G, V, temp_p, temp_q, seed, row_base,
                    out["accept_len"], out["next_token"], out["alpha"], out["beta"], ws,
                    ws.numel(), st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_verify")
    return out


def greedy_select_and_verify(p, drafts, temp_p=1.0, seed=0, row_base=0, want_alpha=False,
                             want_scores=False, workspace=None, stream=None):
    """Greedy acceptance: p [B,K,gamma+1,V] (bf16 or fp32), drafts [B,K,gamma] int32."""
    if stream is not None:
        return _on(stream, p, greedy_select_and_verify, p, drafts, temp_p, seed, row_base,
                   want_alpha, want_scores, workspace)
    import torch
    dev = p.device
    for t, n in ((p, "p"), (drafts, "drafts")):
        _check(t, n, dev)
    if drafts.dtype != torch.int32:
        raise TypeError("drafts must be int32")
    if p.dim() != 4 or drafts.dim() != 3:
        raise ValueError("expected p [B,K,G+1,V], drafts [B,K,G]")
    B, K, G1, V = p.shape
    G = G1 - 1
    if tuple(drafts.shape) != (B, K, G):
        raise ValueError("shape mismatch: p %s drafts %s" % (tuple(p.shape), tuple(drafts.shape)))
    out = {
        "selected": torch.empty(B, dtype=torch.int32, device=dev),
        "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
        "next_token": torch.empty(B, dtype=torch.int32, device=dev),
        "scores": torch.empty((B, K), dtype=torch.float32, device=dev) if want_scores else None,
        "alpha": torch.empty((B, K, G), dtype=torch.float32, device=dev) if want_alpha else None,
    }
    ws = alloc_workspace(B, K, G, V, dev) if workspace is None else workspace
    _check(ws, "workspace", dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    rc = svd_greedy_select_and_verify(p, drafts, _dtype_code(p), B, K, G, V, temp_p, seed,
                                      row_base, out["selected"], out["accept_len"],
                                      out["next_token"], out["scores"], out["alpha"], ws,
                                      ws.numel(), st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_greedy_select_and_verify")
    return out


def greedy_verify(p, draft, temp_p=1.0, seed=0, row_base=0, want_alpha=False, workspace=None,
                  stream=None):
    """Greedy acceptance, one draft: p [B,gamma+1,V] (bf16 or fp32), draft [B,gamma] int32."""
    if stream is not None:
        return _on(stream, p, greedy_verify, p, draft, temp_p, seed, row_base, want_alpha,
                   workspace)
    import torch
    dev = p.device
    for t, n in ((p, "p"), (draft, "draft")):
        _check(t, n, dev)
    if draft.dtype != torch.int32:
        raise TypeError("draft must be int32")
    B, G1, V = p.shape
    G = G1 - 1
    if tuple(draft.shape) != (B, G):
        raise ValueError("shape mismatch")
    out = {
        "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
        "next_token": torch.empty(B, dtype=torch.int32, device=dev),
        "alpha": torch.empty((B, G), dtype=torch.float32, device=dev) if want_alpha else None,
    }
    ws = alloc_workspace(B, 1, G, V, dev) if workspace is None else workspace
    _check(ws, "workspace", dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    rc = svd_greedy_verify(p, draft, _dtype_code(p), B, G, V, temp_p, seed, row_base,
                           out["accept_len"], out["next_token"], out["alpha"], ws, ws.numel(), st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_greedy_verify")
    return out


def select_and_verify_rows(p_pool, p_index, q_pool, q_index, drafts, rule="standard", temp_p=1.0,
                           temp_q=None, seed=0, row_base=0, want_alpha=False, want_scores=False,
                           workspace=None, stream=None):
    """Shared rows: p_pool [NP,V], p_index [B,K,gamma+1] int32, q_pool [NQ,V] and
    q_index [B,K,gamma] int32 (None for rule="greedy"), drafts [B,K,gamma] int32."""
    if stream is not None:
        return _on(stream, p_pool, select_and_verify_rows, p_pool, p_index, q_pool, q_index, drafts,
                   rule, temp_p, temp_q, seed, row_base, want_alpha, want_scores, workspace)
    import torch
    greedy = rule == "greedy"
    if rule not in ("standard", "greedy"):
        raise ValueError("rule must be 'standard' or 'greedy'")
    dev = p_pool.device
    tens = [(p_pool, "p_pool"), (p_index, "p_index"), (drafts, "drafts")]
    if not greedy:
        tens += [(q_pool, "q_pool"), (q_index, "q_index")]
        if q_pool.dtype != p_pool.dtype:
            raise TypeError("p_pool and q_pool must share one dtype")
    for t, n in tens:
        _check(t, n, dev)
    for t, n in ((p_index, "p_index"), (drafts, "drafts")) + (() if greedy else ((q_index, "q_index"),)):
        if t.dtype != torch.int32:
            raise TypeError("%s must be int32" % n)
    B, K, G = drafts.shape
    V = p_pool.shape[1]
    if tuple(p_index.shape) != (B, K, G + 1) or (not greedy and tuple(q_index.shape) != (B, K, G)):
        raise ValueError("index tables must be [B,K,gamma+1] and [B,K,gamma]")
    if not greedy and q_pool.shape[1] != V:
        raise ValueError("pools must share V")
    NP = p_pool.shape[0]
    NQ = 0 if greedy else q_pool.shape[0]
    out = {
        "selected": torch.empty(B, dtype=torch.int32, device=dev),
        "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
        "next_token": torch.empty(B, dtype=torch.int32, device=dev),
        "scores": torch.empty((B, K), dtype=torch.float32, device=dev) if want_scores else None,
        "alpha": torch.empty((B, K, G), dtype=torch.float32, device=dev) if want_alpha else None,
    }
    if workspace is None:
        n = svd_rows_workspace_bytes(B, K, G, V, NP, NQ)
        if n == 0:
            raise ValueError("sizes out of range")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    temp_q = temp_p if temp_q is None else temp_q
    rc = svd_select_and_verify_rows(
        SVD_RULE_GREEDY if greedy else SVD_RULE_STANDARD, p_pool, NP, p_index,
        None if greedy else q_pool, NQ, None if greedy else q_index, drafts, _dtype_code(p_pool),
        B, K, G, V, temp_p, temp_q, seed, row_base, out["selected"], out["accept_len"],
        out["next_token"], out["scores"], out["alpha"], workspace, workspace.numel(), st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_select_and_verify_rows")
    return out


def verify_window(p, q, drafts, gamma_b=None, eos=-1, rule="standard", early_exit=False,
                  temp_p=1.0, temp_q=None, seed=0, row_base=0, want_alpha=False,
                  want_scores=False, workspace=None, stream=None):
    """Ragged, EOS-aware windows: p [B,K,gamma+1,V], q [B,K,gamma,V] (None for
    rule="greedy"), drafts [B,K,gamma] int32, gamma_b [B] int32 or None, eos a token or -1.
    early_exit (K = 1): stream positions only up to each prefix's first rejection."""
    if stream is not None:
        return _on(stream, p, verify_window, p, q, drafts, gamma_b, eos, rule, early_exit, temp_p,
                   temp_q, seed, row_base, want_alpha, want_scores, workspace)
    import torch
    greedy = rule == "greedy"
    if rule not in ("standard", "greedy"):
        raise ValueError("rule must be 'standard' or 'greedy'")
    dev = p.device
    tens = [(p, "p"), (drafts, "drafts")] + ([] if greedy else [(q, "q")])
    if gamma_b is not None:
        tens.append((gamma_b, "gamma_b"))
    for t, n in tens:
        _check(t, n, dev)
    B, K, G1, V = p.shape
    G = G1 - 1
    if tuple(drafts.shape) != (B, K, G) or (gamma_b is not None and tuple(gamma_b.shape) != (B,)):
        raise ValueError("drafts must be [B,K,gamma] and gamma_b [B]")
    out = {
        "selected": torch.empty(B, dtype=torch.int32, device=dev),
        "accept_len": torch.empty(B, dtype=torch.int32, device=dev),
        "next_token": torch.empty(B, dtype=torch.int32, device=dev),
        "scores": torch.empty((B, K), dtype=torch.float32, device=dev) if want_scores else None,
        "alpha": torch.empty((B, K, G), dtype=torch.float32, device=dev) if want_alpha else None,
    }
    ws = alloc_workspace(B, K, G, V, dev) if workspace is None else workspace
    _check(ws, "workspace", dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    temp_q = temp_p if temp_q is None else temp_q
    rc = svd_verify_window(SVD_RULE_GREEDY if greedy else SVD_RULE_STANDARD, p,
                           None if greedy else q, drafts, gamma_b, eos, int(bool(early_exit)),
                           _dtype_code(p), B, K, G, V, temp_p, temp_q, seed, row_base,
                           out["selected"], out["accept_len"], out["next_token"], out["scores"],
                           out["alpha"], ws, ws.numel(), st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_verify_window")
    return out


def cps_lattice(q, temp_q=1.0, tau=0.8, m_max=15, eos=-1, stream=None, lib=None):
    """Candidate lattice of drafter logits q [B, G, V] (bf16 or fp32); lib: the
    Library to call (default: the product library)."""
    if stream is not None:
        return _on(stream, q, cps_lattice, q, temp_q, tau, m_max, eos, None, lib)
    import torch
    dev = q.device
    _check(q, "q", dev)
    B, G, V = q.shape
    out = {"cand": torch.empty((B, G, m_max), dtype=torch.int32, device=dev),
           "cand_logp": torch.empty((B, G, m_max), dtype=torch.float32, device=dev),
           "n_cand": torch.empty((B, G), dtype=torch.int32, device=dev),
           "len": torch.empty(B, dtype=torch.int32, device=dev)}
    n = svd_cps_workspace_bytes(B, G)
    if n == 0:
        raise ValueError("sizes out of range")
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    lib = _default if lib is None else lib
    rc = lib.svd_cps_lattice(q, _dtype_code(q), B, G, V, temp_q, tau, m_max, eos, out["cand"],
                             out["cand_logp"], out["n_cand"], out["len"], ws, n, st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_cps_lattice")
    return out


def cps_beam(lat, fluency=None, lam=1.0, beam=3, stream=None, lib=None):
    """Beam search over a lattice from cps_lattice; fluency [B, G, m_max, m_max] fp32 or None;
    lib: the Library to call (default: the product library)."""
    if stream is not None:
        return _on(stream, lat["cand"], cps_beam, lat, fluency, lam, beam, None, lib)
    import torch
    cand = lat["cand"]
    dev = cand.device
    B, G, M = cand.shape
    if fluency is not None:
        _check(fluency, "fluency", dev)
        if fluency.dtype != torch.float32 or tuple(fluency.shape) != (B, G, M, M):
            raise ValueError("fluency must be float32 [B, G, m_max, m_max]")
    out = {"paths": torch.empty((B, beam, G), dtype=torch.int32, device=dev),
           "score": torch.empty((B, beam), dtype=torch.float32, device=dev),
           "path_len": torch.empty((B, beam), dtype=torch.int32, device=dev)}
    st = torch.cuda.current_stream(dev).cuda_stream
    lib = _default if lib is None else lib
    rc = lib.svd_cps_beam(cand, lat["cand_logp"], lat["n_cand"], lat["len"], fluency, lam, B, G,
                          M, beam, out["paths"], out["score"], out["path_len"], st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_cps_beam")
    return out


def adl_next(drafts, selected, accept_len, avg, gamma_b=None, eos=-1, k_min=1, k_max=64, step=4,
             shift=2, slack=64, stream=None):
    """Adaptive draft length: the next window of every prefix, on the device.
    drafts [B,K,gamma] int32 and selected, accept_len [B] int32 (a verification
    call's inputs and outputs), gamma_b [B] int32 or None, avg [B,2] int32
    updated in place.  Returns next [B] int32."""
    if stream is not None:
        return _on(stream, drafts, adl_next, drafts, selected, accept_len, avg, gamma_b, eos, k_min,
                   k_max, step, shift, slack)
    import torch
    dev = drafts.device
    tens = [(drafts, "drafts"), (selected, "selected"), (accept_len, "accept_len"),
            (avg, "avg")] + ([] if gamma_b is None else [(gamma_b, "gamma_b")])
    for t, n in tens:
        _check(t, n, dev)
        if t.dtype != torch.int32:
            raise TypeError("%s must be int32" % n)
    B, K, G = drafts.shape
    if (tuple(selected.shape) != (B,) or tuple(accept_len.shape) != (B,) or
            tuple(avg.shape) != (B, 2) or (gamma_b is not None and tuple(gamma_b.shape) != (B,))):
        raise ValueError("selected, accept_len, gamma_b must be [B] and avg [B, 2]")
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    st = torch.cuda.current_stream(dev).cuda_stream
    rc = svd_adl_next(drafts, selected, accept_len, gamma_b, eos, B, K, G, k_min, k_max, step,
                      shift, slack, avg, nxt, st)
    if rc != SVD_OK:
        raise SvdError(rc, "svd_adl_next")
    return nxt


# --------------------------------------------------------------------------
# Around the verification step: the draft tree, the paged cache, the attention
# of the tree over it, and the adjustments of the verifier's logits.
#
# A decode step makes these calls on small tensors, where the host's share is
# what counts: one check per tensor, pointers passed as they are, the current
# stream's handle taken without a Stream object.

def _bad(t, name, dev, dtype, shape):
    """Say what is wrong with a tensor that failed its check."""
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d" % (name, dev))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _ptr(t, name, dev, dtype, shape):
    """Address of a contiguous tensor of this device (its index), dtype and shape, or None."""
    if t is None:
        return None
    if (t.get_device() != dev or t.dtype != dtype or t.shape != shape or
            not t.is_contiguous()):
        _bad(t, name, dev, dtype, shape)
    return t.data_ptr()


def _workspace(t, dev):
    """(address, bytes) of a caller's workspace on this device (its index)."""
    if t.get_device() != dev:
        raise ValueError("workspace must be on cuda:%d" % dev)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _device_of(t, name):
    """Index of the GPU that a tensor is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be on the GPU" % name)
    return dev


def _call(f, name, dev, *args):
    """f(*args, the current stream) with dev as the current device."""
    C = _T._C
    stream = C._cuda_getCurrentRawStream(dev)
    if C._cuda_getDevice() == dev:
        rc = f(*args, stream)
    else:
        with _T.cuda.device(dev):
            rc = f(*args, stream)
    if rc != SVD_OK:
        raise SvdError(rc, name)


def draft_tree(drafts, root=None, n_max=None, stream=None):
    """The prefix tree of drafts [B,K,gamma] int32: root [B] int32 the last
    committed tokens, n_max room for nodes (default 1 + K * gamma, which always
    suffices).  Returns tokens, parent, depth [B,n_max], anc [B,n_max,W] (bit i % 32
    of word i // 32: node i is on the node's path), n_nodes [B] and p_index
    [B,K,gamma+1], the rows of the pool [B * n_max, V] for select_and_verify_rows (which
    takes whole drafts: one that ends early, at a negative token, gives its prefix -1)."""
    if stream is not None:
        return _on(stream, drafts, draft_tree, drafts, root, n_max)
    torch = _torch()
    dev, i32 = _device_of(drafts, "drafts"), torch.int32
    if drafts.dim() != 3:
        raise ValueError("drafts must be [B,K,gamma]")
    B, K, G = drafts.shape
    d = _ptr(drafts, "drafts", dev, i32, drafts.shape)
    r = _ptr(root, "root", dev, i32, (B,))
    T = 1 + K * G if n_max is None else int(n_max)
    W = (T + 31) // 32
    BT, P = B * T, K * (G + 1)
    # one allocation: tokens, parent, depth, anc, p_index, n_nodes
    o1, o2, o3 = BT, 2 * BT, 3 * BT
    o4 = o3 + BT * W
    o5 = o4 + B * P
    flat = torch.empty(max(o5 + B, 0), dtype=i32, device=dev)
    at = flat.data_ptr()
    _call(_c.svd_draft_tree, "svd_draft_tree", dev, d, r, B, K, G, T, at, at + 4 * o1,
          at + 4 * o2, at + 4 * o3, at + 4 * o5, at + 4 * o4)
    view = flat.as_strided
    return {"tokens": view((B, T), (T, 1)), "parent": view((B, T), (T, 1), o1),
            "depth": view((B, T), (T, 1), o2), "anc": view((B, T, W), (T * W, W, 1), o3),
            "n_nodes": view((B,), (1,), o5), "p_index": view((B, K, G + 1), (P, G + 1, 1), o4)}


def kv_cache(n_pages, kv_heads, page, head_dim, dtype=None, device="cuda"):
    """An empty paged cache: k and v [n_pages,kv_heads,page,head_dim] of
    torch.bfloat16 (the default) or torch.float8_e4m3fn, and for the latter
    k_scale and v_scale [n_pages,kv_heads,page] uint8 (exponent + 127)."""
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError("a cache is torch.bfloat16 or torch.float8_e4m3fn, got %s" % dtype)
    c = {n: torch.zeros((n_pages, kv_heads, page, head_dim), dtype=dtype, device=device)
         for n in ("k", "v")}
    for n in ("k_scale", "v_scale"):
        c[n] = (None if dtype == torch.bfloat16 else
                torch.full((n_pages, kv_heads, page), 127, dtype=torch.uint8, device=device))
    return c


def _cache_struct(cache, block_table, B):
    """(the C struct of a cache and its block table, the device's index)."""
    torch = _torch()
    k, v = cache["k"], cache["v"]
    dev, dtype, shape = _device_of(k, "cache k"), k.dtype, k.shape
    if len(shape) != 4:
        raise ValueError("cache k and v must be [n_pages,kv_heads,page,head_dim]")
    if dtype == torch.float8_e4m3fn:
        code, ks, vs = SVD_CACHE_E4M3, cache["k_scale"], cache["v_scale"]
        ks = _ptr(ks, "cache k_scale", dev, torch.uint8, shape[:3])
        vs = _ptr(vs, "cache v_scale", dev, torch.uint8, shape[:3])
    elif dtype == torch.bfloat16:
        code, ks, vs = SVD_CACHE_BF16, None, None
    else:
        raise TypeError("a cache is torch.bfloat16 or torch.float8_e4m3fn, got %s" % dtype)
    n_pages, heads, page, D = shape
    mp = 0
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B,max_pages]")
        mp = block_table.shape[1]
    return CacheStruct(_ptr(k, "cache k", dev, dtype, shape), _ptr(v, "cache v", dev, dtype, shape),
                       ks, vs, _ptr(block_table, "block_table", dev, torch.int32, (B, mp)),
                       n_pages, mp, page, heads, D, code), dev


def _tokens(t, name, heads, D, dev):
    """Elements between the tokens of t [B,T,heads,D], whose heads are contiguous."""
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d" % (name, dev))
    shape = t.shape
    if len(shape) != 4 or shape[2] != heads or shape[3] != D:
        raise ValueError("%s must be [B,T,%d,%d], got %s" % (name, heads, D, list(shape)))
    if t.is_contiguous():
        return heads * D
    B, T = shape[:2]
    sb, st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (heads > 1 and sh != D):
        raise ValueError("the heads of a token of %s must be contiguous" % name)
    if T == 1:
        st = sb if B > 1 else heads * D
    elif B > 1 and sb != T * st:
        raise ValueError("the tokens of %s must be evenly strided" % name)
    return st


def cache_write(cache, k, v, block_table, ctx_len, n_new=None, dst=None, stream=None):
    """Write k, v [B,T,kv_heads,D] (bf16 or fp32; the tokens may be strided, as in
    a fused projection) to positions ctx_len[b] + t, or ctx_len[b] + dst[b,t] where
    dst is not negative; n_new [B] limits the tokens of a sequence.  cache: as from
    kv_cache; block_table [B,max_pages], ctx_len [B], dst [B,T] int32."""
    if stream is not None:
        return _on(stream, k, cache_write, cache, k, v, block_table, ctx_len, n_new, dst)
    i32 = _torch().int32
    B, T = k.shape[:2]
    c, dev = _cache_struct(cache, block_table, B)
    ks = _tokens(k, "k", c.kv_heads, c.head_dim, dev)
    vs = _tokens(v, "v", c.kv_heads, c.head_dim, dev)
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must share one shape and dtype")
    _call(_c.svd_cache_write, "svd_cache_write", dev, ctypes.addressof(c), k.data_ptr(),
          v.data_ptr(), _dtype_code(k), ks, vs, _ptr(ctx_len, "ctx_len", dev, i32, (B,)),
          _ptr(n_new, "n_new", dev, i32, (B,)), _ptr(dst, "dst", dev, i32, (B, T)), B, T)


def cache_read(cache, block_table, n, start=None, count=None, dtype=None, out=None, stream=None):
    """Positions start[b] .. start[b] + n - 1 of every sequence as (k, v), each
    [B,n,kv_heads,D] of dtype (default torch.bfloat16, or torch.float32).  count
    [B] limits a sequence; the rows behind it are left as out = (k, v) has them."""
    if stream is not None:
        return _on(stream, block_table, cache_read, cache, block_table, n, start, count, dtype, out)
    torch = _torch()
    i32 = torch.int32
    B = block_table.shape[0]
    c, dev = _cache_struct(cache, block_table, B)
    shape = (B, n, c.kv_heads, c.head_dim)
    if out is None:
        both = torch.empty((2,) + shape, dtype=torch.bfloat16 if dtype is None else dtype,
                           device=dev)
        k, v = both.unbind()
    else:
        k, v = out
        if k.dtype != v.dtype or (dtype is not None and k.dtype != dtype):
            raise TypeError("out k and v must share the asked dtype")
    _call(_c.svd_cache_read, "svd_cache_read", dev, ctypes.addressof(c),
          _ptr(start, "start", dev, i32, (B,)), _ptr(count, "count", dev, i32, (B,)), B, n,
          _dtype_code(k), _ptr(k, "out k", dev, k.dtype, shape),
          _ptr(v, "out v", dev, k.dtype, shape))
    return k, v


def tree_attention_workspace(B, T, q_heads, cache, block_table):
    """A workspace for tree_attention calls of these sizes."""
    torch = _torch()
    k = cache["k"]
    n = svd_tree_attention_workspace_bytes(B, T, q_heads, k.shape[1], k.shape[3],
                                           block_table.shape[1] * k.shape[2])
    if n == 0:
        raise ValueError("sizes out of range: B=%d T=%d q_heads=%d cache %s" %
                         (B, T, q_heads, list(k.shape)))
    return torch.empty(n, dtype=torch.uint8, device=k.device)


def tree_attention(q, cache, block_table, ctx_len, anc=None, n_nodes=None, scale=None, out=None,
                   lse=None, want_lse=False, workspace=None, stream=None):
    """q [B,T,q_heads,D] bf16 (the tokens may be strided) over the cache: node t of
    sequence b attends to the ctx_len[b] cached tokens and the nodes of anc[b,t]
    (None: a chain, nodes 0..t), whose keys and values cache_write has put at
    positions ctx_len[b] + node.  scale: default D ** -0.5.  Returns out
    [B,T,q_heads,D] bf16 and, when asked for or given, lse [B,T,q_heads] fp32; rows
    from n_nodes[b] on are left as out and lse have them."""
    if stream is not None:
        return _on(stream, q, tree_attention, q, cache, block_table, ctx_len, anc, n_nodes, scale,
                   out, lse, want_lse, workspace)
    torch = _torch()
    i32, bf16 = torch.int32, torch.bfloat16
    if q.dtype != bf16:
        raise TypeError("q must be bfloat16, got %s" % q.dtype)
    if q.dim() != 4:
        raise ValueError("q must be [B,T,q_heads,D]")
    B, T, Hq, D = q.shape
    c, dev = _cache_struct(cache, block_table, B)
    qs = _tokens(q, "q", Hq, c.head_dim, dev)
    if Hq % c.kv_heads != 0:
        raise ValueError("q_heads must be a multiple of the cache's kv_heads")
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=bf16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = tree_attention_workspace(B, T, Hq, cache, block_table)
    ws, ws_bytes = _workspace(workspace, dev)
    _call(_c.svd_tree_attention, "svd_tree_attention", dev, ctypes.addressof(c),
          q.data_ptr(), qs, _ptr(ctx_len, "ctx_len", dev, i32, (B,)),
          _ptr(n_nodes, "n_nodes", dev, i32, (B,)),
          _ptr(anc, "anc", dev, i32, (B, T, (T + 31) // 32)),
          D ** -0.5 if scale is None else scale, B, T, Hq,
          _ptr(out, "out", dev, bf16, (B, T, Hq, D)),
          _ptr(lse, "lse", dev, torch.float32, (B, T, Hq)), ws, ws_bytes)
    return {"out": out, "lse": lse}


def adjust_logits(logits, history=None, hist_len=None, prompt_len=None, tokens=None, anc=None,
                  n_rows=None, repetition=None, frequency=None, presence=None, bias=None,
                  allow=None, allow_index=None, out=None, stream=None):
    """Penalties, biases and grammar masks on logits [B,T,V] (bf16 or fp32), row
    (b, t) after node t of a tree.  history [B,H] int32 with hist_len [B] tokens
    used (prompt_len [B] of them the prompt), tokens [B,T] and anc [B,T,W] of the
    tree (the root counts as generated: the history does not hold it, too);
    repetition, frequency, presence [B] fp32; bias = (offsets [B+1] int32, tokens
    int32, values fp32); allow [n,ceil(V/32)] int32 bit masks and allow_index [B,T]
    int32 (negative: none).  out: default a new tensor; logits itself for a change in
    place.  Returns out."""
    if stream is not None:
        return _on(stream, logits, adjust_logits, logits, history, hist_len, prompt_len, tokens,
                   anc, n_rows, repetition, frequency, presence, bias, allow, allow_index, out)
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    if logits.dim() != 3:
        raise ValueError("logits must be [B,T,V]")
    dev, dtype, shape = _device_of(logits, "logits"), logits.dtype, logits.shape
    z = _ptr(logits, "logits", dev, dtype, shape)
    B, T, V = shape
    b, bt = (B,), (B, T)
    H, h = 0, None
    if history is not None:
        if history.dim() != 2 or hist_len is None:
            raise ValueError("history must be [B,H], with hist_len")
        H = history.shape[1]
        h = _ptr(history, "history", dev, i32, (B, H)) if H else None
    off = tok = val = None
    n_bias = 0
    if bias is not None:
        off, tok, val = bias
        n_bias = tok.numel()
        off = _ptr(off, "bias offsets", dev, i32, (B + 1,))
        tok = _ptr(tok, "bias tokens", dev, i32, (n_bias,))
        val = _ptr(val, "bias values", dev, f32, (n_bias,))
    n_masks = 0
    if allow is not None:
        if allow.dim() != 2 or allow_index is None:
            raise ValueError("allow must be [n,ceil(V/32)], with allow_index")
        n_masks = allow.shape[0]
        allow = _ptr(allow, "allow", dev, i32, (n_masks, (V + 31) // 32))
    if out is None:
        out = torch.empty_like(logits)
    _call(_c.svd_adjust_logits, "svd_adjust_logits", dev, z,
          _ptr(out, "out", dev, dtype, shape), _dtype_code(logits), B, T, V,
          _ptr(n_rows, "n_rows", dev, i32, b), h, H, _ptr(hist_len, "hist_len", dev, i32, b),
          _ptr(prompt_len, "prompt_len", dev, i32, b), _ptr(tokens, "tokens", dev, i32, bt),
          _ptr(anc, "anc", dev, i32, (B, T, (T + 31) // 32)),
          _ptr(repetition, "repetition", dev, f32, b), _ptr(frequency, "frequency", dev, f32, b),
          _ptr(presence, "presence", dev, f32, b), off, tok, val, n_bias, allow,
          _ptr(allow_index, "allow_index", dev, i32, bt), n_masks)
    return out


# --------------------------------------------------------------------------
# A serving loop's other operators: block tables and slot maps of the cache,
# filtered and sampled logits, attention over shared prefixes.

def page_pool(n_pages, B, max_pages, device="cuda"):
    """The block tables of B empty sequences and a ring of n_pages free pages: table
    [B,max_pages], held [B] entries in use, free [n_pages], state [2] = the ring's
    first place and its count; all int32."""
    torch = _torch()
    i32 = dict(dtype=torch.int32, device=device)
    return {"table": torch.full((B, max_pages), -1, **i32), "held": torch.zeros(B, **i32),
            "free": torch.arange(n_pages, **i32), "state": torch.tensor([0, n_pages], **i32)}


def cache_pages(pool, length, page, shared=None, out=None, workspace=None, stream=None):
    """Give every sequence the pages that length [B] int32 tokens need: a sequence that
    grows takes pages from the head of the ring, in sequence order, one that shrinks gives
    its last ones back behind the ring's end, where later calls find them.  shared [B]:
    the first shared[b] entries belong to others and are never given back.  pool: as from
    page_pool, changed in place; with out = {"table", "held", "state"} these are written
    instead, and of pool only free[...] behind the ring's end.  Returns room [B] int32,
    the tokens that a sequence has pages for: less than length where the ring had too few
    (nothing of it has changed then), -1 where its length, held or shared is out of range,
    or the ring's state is."""
    if stream is not None:
        return _on(stream, length, cache_pages, pool, length, page, shared, out, workspace)
    torch = _torch()
    i32 = torch.int32
    table = pool["table"]
    dev = _device_of(table, "pool table")
    if table.dim() != 2 or pool["free"].dim() != 1:
        raise ValueError("pool table must be [B,max_pages] and pool free [n_pages]")
    B, mp = table.shape
    n = pool["free"].shape[0]
    to = pool if out is None else out
    p, o = ([_ptr(d[k], what + " " + k, dev, i32, s)
             for k, s in (("state", (2,)), ("held", (B,)), ("table", (B, mp)))]
            for d, what in ((pool, "pool"), (to, "out")))
    if workspace is None:
        # the results and the plan in one allocation
        both = torch.empty((4 * B + 255) // 256 * 256 + svd_cache_pages_workspace_bytes(B),
                           dtype=torch.uint8, device=table.device)
        room = both[:4 * B].view(i32)
        ws, ws_bytes = both.data_ptr() + (4 * B + 255) // 256 * 256, both.numel()
        ws_bytes -= (4 * B + 255) // 256 * 256
    else:
        room = torch.empty(B, dtype=i32, device=table.device)
        ws, ws_bytes = _workspace(workspace, dev)
    _call(_c.svd_cache_pages, "svd_cache_pages", dev, _ptr(length, "length", dev, i32, (B,)),
          _ptr(shared, "shared", dev, i32, (B,)), B, mp, page, n,
          _ptr(pool["free"], "pool free", dev, i32, (n,)), *p, *o, room.data_ptr(), ws, ws_bytes)
    return room


def cache_slots(cache, block_table, ctx_len, n_new, n, stream=None):
    """Where packed tokens go: sequence b brings n_new[b] tokens behind its ctx_len[b], the
    sequences one after another in n places.  Returns row_off [B+1] int32, where each
    sequence begins, and for every place seq, pos [n] int32 and slot [n] int64, the
    token's sequence, its position, and page * (tokens a page) + place, for
    cache_write_slots; all -1 behind the last token, slot alone where a position has no
    page."""
    if stream is not None:
        return _on(stream, block_table, cache_slots, cache, block_table, ctx_len, n_new, n)
    torch = _torch()
    i32 = torch.int32
    dev = _device_of(block_table, "block_table")
    if block_table.dim() != 2 or cache["k"].dim() != 4:
        raise ValueError("block_table must be [B,max_pages], cache k [n_pages,kv_heads,page,D]")
    B, mp = block_table.shape
    n_pages, _, page, _ = cache["k"].shape
    # one allocation: slot, then seq, pos, row_off
    flat = torch.empty(max(n + (2 * n + B + 2) // 2, 0), dtype=torch.int64, device=block_table.device)
    at = flat.data_ptr()
    _call(_c.svd_cache_slots, "svd_cache_slots", dev, _ptr(ctx_len, "ctx_len", dev, i32, (B,)),
          _ptr(n_new, "n_new", dev, i32, (B,)), _ptr(block_table, "block_table", dev, i32, (B, mp)),
          B, mp, page, n_pages, n, at + 16 * n, at + 8 * n, at + 12 * n, at)
    view = flat.view(i32).as_strided
    return {"row_off": view((B + 1,), (1,), 4 * n), "seq": view((n,), (1,), 2 * n),
            "pos": view((n,), (1,), 3 * n), "slot": flat[:n]}


def _packed(t, name, heads, D, dev):
    """Elements between the tokens of t [n,heads,D], whose heads are contiguous."""
    if t.dim() != 3:
        raise ValueError("%s must be [n,%d,%d], got %s" % (name, heads, D, list(t.shape)))
    return _tokens(t.unsqueeze(0), name, heads, D, dev)


def cache_write_slots(cache, k, v, slot, stream=None):
    """Write packed k, v [n,kv_heads,D] (bf16 or fp32; the tokens may be strided) to slot
    [n] int64, as from cache_slots; a slot outside the pages is skipped."""
    if stream is not None:
        return _on(stream, k, cache_write_slots, cache, k, v, slot)
    torch = _torch()
    c, dev = _cache_struct(cache, None, 0)
    ks = _packed(k, "k", c.kv_heads, c.head_dim, dev)
    vs = _packed(v, "v", c.kv_heads, c.head_dim, dev)
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must share one shape and dtype")
    n = k.shape[0]
    _call(_c.svd_cache_write_slots, "svd_cache_write_slots", dev, ctypes.addressof(c),
          k.data_ptr(), v.data_ptr(), _dtype_code(k), ks, vs,
          _ptr(slot, "slot", dev, torch.int64, (n,)), n)


def _filter_args(logits, n_rows, temperature, top_k, top_p, min_p):
    """(device, pointers and sizes of a filter or sample call up to min_p)."""
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    if logits.dim() != 3:
        raise ValueError("logits must be [B,T,V]")
    dev = _device_of(logits, "logits")
    B, T, V = logits.shape
    b = (B,)
    return (dev, _ptr(logits, "logits", dev, logits.dtype, logits.shape), _dtype_code(logits),
            (B, T, V), (_ptr(n_rows, "n_rows", dev, i32, b),
                        _ptr(temperature, "temperature", dev, f32, b),
                        _ptr(top_k, "top_k", dev, i32, b), _ptr(top_p, "top_p", dev, f32, b),
                        _ptr(min_p, "min_p", dev, f32, b)))


def filter_logits(logits, temperature=None, top_k=None, top_p=None, min_p=None, n_rows=None,
                  out=None, stream=None):
    """logits [B,T,V] (bf16 or fp32) with -inf for the tokens that a prefix's settings drop:
    with weights exp((z - max z) / temperature), min_p keeps those of at least min_p, top_k
    the first top_k of them by falling logit (the lower index first among equal ones; 0 or
    less: all), top_p the shortest beginning of that order that holds top_p of their
    weight.  temperature, top_p, min_p [B] fp32, top_k [B] int32, each or None; a
    temperature of 0 keeps the first most likely token alone.  The logits themselves are
    not divided by the temperature: a verification is lossless for the filtered laws where its
    temp_p (temp_q for a drafter's rows) is the prefix's temperature, and it has one for its
    batch, so prefixes of other temperatures go to calls of their own, or fp32 logits are
    divided first, filtered without a temperature and verified at 1.  n_rows [B]: rows from
    n_rows[b] on are left as out has them.  out: default a new tensor; logits itself for a change in place.  Returns out."""
    if stream is not None:
        return _on(stream, logits, filter_logits, logits, temperature, top_k, top_p, min_p, n_rows,
                   out)
    dev, z, code, (B, T, V), ask = _filter_args(logits, n_rows, temperature, top_k, top_p, min_p)
    if out is None:
        out = _torch().empty_like(logits)
    _call(_c.svd_filter_logits, "svd_filter_logits", dev, z,
          _ptr(out, "out", dev, logits.dtype, logits.shape), code, B, T, V, *ask)
    return out


def sample(logits, uniforms=None, K=1, temperature=None, top_k=None, top_p=None, min_p=None,
           n_rows=None, seed=0, row_base=0, token=None, logprob=None, want_logprob=False,
           stream=None):
    """K tokens from every row of logits [B,T,V], among those that filter_logits keeps, by
    the softmax at the temperature: the first token, by index, up to which the kept
    weights exceed uniforms times their sum.  uniforms [B,K,T] fp64 in [0,1) (K follows
    from it); None: the library's counter hash of seed, row_base + b and k * T + t.
    Returns token [B,K,T] int32 (-1 for a row without an answer) and, when asked for or
    given, logprob [B,K,T] fp32, the logarithm of the token's share of the kept weight;
    rows from n_rows[b] on are left as token and logprob have them."""
    if stream is not None:
        return _on(stream, logits, sample, logits, uniforms, K, temperature, top_k, top_p, min_p,
                   n_rows, seed, row_base, token, logprob, want_logprob)
    torch = _torch()
    dev, z, code, (B, T, V), ask = _filter_args(logits, n_rows, temperature, top_k, top_p, min_p)
    if uniforms is not None:
        if uniforms.dim() != 3:
            raise ValueError("uniforms must be [B,K,T]")
        K = uniforms.shape[1]
    shape = (B, K, T)
    if token is None:
        token = torch.empty(shape, dtype=torch.int32, device=logits.device)
    if logprob is None and want_logprob:
        logprob = torch.empty(shape, dtype=torch.float32, device=logits.device)
    _call(_c.svd_sample, "svd_sample", dev, z, code, B, T, V, K, *ask,
          _ptr(uniforms, "uniforms", dev, torch.float64, shape), int(seed) & _M64,
          int(row_base) & _M64, _ptr(token, "token", dev, torch.int32, shape),
          _ptr(logprob, "logprob", dev, torch.float32, shape))
    return {"token": token, "logprob": logprob}


def prefix_attention_workspace(B, T, q_heads, cache, block_table, n_groups=0):
    """A workspace for prefix_attention calls of these sizes."""
    torch = _torch()
    k = cache["k"]
    n = svd_prefix_attention_workspace_bytes(B, T, q_heads, k.shape[1], k.shape[3],
                                             block_table.shape[1] * k.shape[2], n_groups)
    if n == 0:
        raise ValueError("sizes out of range: B=%d T=%d q_heads=%d cache %s groups=%d" %
                         (B, T, q_heads, list(k.shape), n_groups))
    return torch.empty(n, dtype=torch.uint8, device=k.device)


def prefix_attention(q, cache, block_table, ctx_len, share_off=None, anc=None, n_nodes=None,
                     depth=None, scale=None, cap=0.0, slopes=None, out=None, lse=None,
                     want_lse=False, workspace=None, stream=None):
    """tree_attention for batches that share prefixes, and for scores that are capped or
    fall off with distance.  share_off [groups+1] int32: sequences share_off[g] to
    share_off[g+1] - 1 are a group, and the pages that all of their block tables begin
    with are read once for the group; what is computed does not depend on it (few sequences,
    or few shared tokens, are faster without).  cap: scores
    become cap * tanh(score / cap) (0 or None: as they are; 16384 at most).  slopes [q_heads] fp32: a
    score loses slopes[h] times the distance between the two positions, a node's position
    being ctx_len[b] + its depth (depth [B,T] int32, needed with anc).  The rest as for
    tree_attention."""
    if stream is not None:
        return _on(stream, q, prefix_attention, q, cache, block_table, ctx_len, share_off, anc,
                   n_nodes, depth, scale, cap, slopes, out, lse, want_lse, workspace)
    torch = _torch()
    i32, bf16, f32 = torch.int32, torch.bfloat16, torch.float32
    if q.dtype != bf16:
        raise TypeError("q must be bfloat16, got %s" % q.dtype)
    if q.dim() != 4:
        raise ValueError("q must be [B,T,q_heads,D]")
    B, T, Hq, D = q.shape
    c, dev = _cache_struct(cache, block_table, B)
    qs = _tokens(q, "q", Hq, c.head_dim, dev)
    if Hq % c.kv_heads != 0:
        raise ValueError("q_heads must be a multiple of the cache's kv_heads")
    G = 0
    if share_off is not None:
        if share_off.dim() != 1 or share_off.shape[0] < 2:
            raise ValueError("share_off must be [groups+1]")
        G = share_off.shape[0] - 1
    if slopes is not None and anc is not None and depth is None:
        raise ValueError("slopes over a tree need its depth")
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=bf16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, T, Hq), dtype=f32, device=dev)
    if workspace is None:
        workspace = prefix_attention_workspace(B, T, Hq, cache, block_table, G)
    ws, ws_bytes = _workspace(workspace, dev)
    _call(_c.svd_prefix_attention, "svd_prefix_attention", dev, ctypes.addressof(c),
          q.data_ptr(), qs, _ptr(ctx_len, "ctx_len", dev, i32, (B,)),
          _ptr(n_nodes, "n_nodes", dev, i32, (B,)),
          _ptr(anc, "anc", dev, i32, (B, T, (T + 31) // 32)),
          _ptr(depth, "depth", dev, i32, (B, T)), _ptr(share_off, "share_off", dev, i32, (G + 1,)),
          G, D ** -0.5 if scale is None else scale, cap or 0.0,
          _ptr(slopes, "slopes", dev, f32, (Hq,)), B, T, Hq,
          _ptr(out, "out", dev, bf16, (B, T, Hq, D)), _ptr(lse, "lse", dev, f32, (B, T, Hq)), ws,
          ws_bytes)
    return {"out": out, "lse": lse}
