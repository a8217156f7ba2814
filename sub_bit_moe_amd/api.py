"""Python front end of libsbm: argument marshalling only.

Every step of the codec and of the fused decode + matvec runs in libsbm.so
(host C++ for dictionary/encoding, HIP kernels on the GPU).  numpy arrays are
used for host buffers, torch tensors for device memory and streams.

A call with stream= runs on that stream, which has to have waited for whatever
wrote the call's inputs, and these have to be kept until it has read them.
Results and workspaces that the call makes belong to that stream; another one
waits for it before it reads them.
"""
from __future__ import annotations

import ctypes as C
import struct
import threading
from dataclasses import dataclass

import numpy as np

from . import _native as N
from ._native import check, lib


def _ptr(a) -> int:
    if a is None:
        return 0
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return int(a.data_ptr())


_current_stream = None


def _stream(stream=None, at=None) -> int:
    """The stream's handle; of the current stream without building a Stream object (2.6 us) for it.  at: the index of the device
    that the call's tensors are on, which has to be the stream's."""
    if stream is not None:
        if at is not None and stream.device_index != at:
            raise ValueError(f"the tensors are on device {at}, the stream on device {stream.device_index}")
        return int(stream.cuda_stream)
    global _current_stream
    if _current_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if raw is None or device is None:
            _current_stream = (lambda d: int(torch.cuda.current_stream(d).cuda_stream)), torch.cuda.current_device
        else:
            _current_stream = raw, device
    now = _current_stream[1]()
    if at is not None and now != at:
        raise ValueError(f"the tensors are on device {at}, the current device is {now}")
    return _current_stream[0](now)


def _made_on(stream, make, *args, **kw):
    """make(*args, **kw), a tensor that a call on `stream` writes: allocated, and filled, on that stream.  Memory of the
    current stream could still be in use there, or be given out again there before the call has written it.  The serving
    calls, which are bound by the host, come here only with a stream."""
    if stream is None:
        return make(*args, **kw)
    import torch
    with torch.cuda.stream(stream):
        return make(*args, **kw)

# ------------------------------------------------------------------ dictionary

def build_dictionary(p0: float = 0.885):
    """(words uint32[131072], checksum) of the canonical dictionary."""
    words = np.zeros(N.SBM_DICT_WORDS, np.uint32)
    cs = C.c_uint64()
    check(lib().sbm_build_dictionary(C.c_double(p0), words.ctypes.data, C.addressof(cs)))
    return words, int(cs.value)


def dictionary_checksum(words: np.ndarray) -> int:
    words = np.ascontiguousarray(words, np.uint32)
    cs = C.c_uint64()
    check(lib().sbm_dictionary_checksum(words.ctypes.data, C.addressof(cs)))
    return int(cs.value)


def dict_tag(words: np.ndarray) -> int:
    """Dictionary identity carried by every matrix descriptor: the low 32 bits
    of the dictionary's FNV-1a 64 checksum (also in the decode image header)."""
    return dictionary_checksum(words) & 0xFFFFFFFF


def dict_image(words: np.ndarray, slots: int = 3) -> np.ndarray:
    """Compact decode image (uint8 bytes) for the fused kernel: slots=3 for
    tables whose entries hold at most 3 nonzeros (the page's static table),
    slots=4 for tables built for other data (entries with 4 nonzeros)."""
    words = np.ascontiguousarray(words, np.uint32)
    if slots not in (3, 4):
        raise ValueError("slots must be 3 or 4")
    n = int(lib().sbm_dict_image_bytes() if slots == 3 else lib().sbm_dict_image4_bytes())
    out = np.zeros(n, np.uint8)
    fn = lib().sbm_dict_image if slots == 3 else lib().sbm_dict_image4
    check(fn(words.ctypes.data, out.ctypes.data, n))
    return out

# ------------------------------------------------------------------ host codec

def encode_matrix(sym: np.ndarray, words: np.ndarray):
    """Greedy trie encoding of a symbol matrix uint8 [rows, cols] (0/1/2).
    Returns (codes uint16[n], row_off uint32[rows+1], bstart uint32[nblk])."""
    sym = np.ascontiguousarray(sym, np.uint8)
    rows, cols = sym.shape
    words = np.ascontiguousarray(words, np.uint32)
    n = C.c_uint64()
    check(lib().sbm_encode_size(sym.ctypes.data, rows, cols, words.ctypes.data, C.addressof(n)))
    codes = np.zeros(max(int(n.value), 1), np.uint16)
    row_off = np.zeros(rows + 1, np.uint32)
    nblk = (int(n.value) + N.SBM_BLOCK - 1) // N.SBM_BLOCK
    bstart = np.zeros(max(nblk, 1), np.uint32)
    check(lib().sbm_encode_matrix(sym.ctypes.data, rows, cols, words.ctypes.data, codes.ctypes.data,
                                  codes.size, row_off.ctypes.data, bstart.ctypes.data, C.addressof(n)))
    return codes[:int(n.value)], row_off, bstart[:nblk]


def encode_experts(syms, words: np.ndarray):
    """One projection's matrices (same shape, uint8 0/1/2) encoded natively into
    the stack layout: (codes uint16 with aligned bases, row_off uint32
    [E*(rows+1)], bstart uint32, list of MatrixDesc with scale_base = e*rows)."""
    words = np.ascontiguousarray(words, np.uint32)
    syms = [np.ascontiguousarray(m, np.uint8) for m in syms]
    E = len(syms)
    rows, cols = (syms[0].shape if E else (0, 2))
    if any(m.shape != (rows, cols) for m in syms):
        raise ValueError("all matrices of a projection share one shape")
    ptrs = (C.c_void_p * max(E, 1))(*[m.ctypes.data for m in syms])
    nc, nb = C.c_uint64(), C.c_uint64()
    st = lib().sbm_encode_experts(E, ptrs, rows, cols, words.ctypes.data, None, 0, None, None, 0, None,
                                  C.addressof(nc), C.addressof(nb))
    if st not in (0, -6):          # -6: SBM_ENOSPACE, the size query
        check(st)
    codes = np.zeros(max(int(nc.value), 1), np.uint16)
    row_off = np.zeros(max(E * (rows + 1), 1), np.uint32)
    bstart = np.zeros(max(int(nb.value), 1), np.uint32)
    desc = (N.MatrixDesc * max(E, 1))()
    check(lib().sbm_encode_experts(E, ptrs, rows, cols, words.ctypes.data, codes.ctypes.data, codes.size,
                                   row_off.ctypes.data, bstart.ctypes.data, bstart.size, C.addressof(desc),
                                   C.addressof(nc), C.addressof(nb)))
    return codes[:int(nc.value)], row_off[:E * (rows + 1)], bstart[:int(nb.value)], list(desc)[:E]


def block_starts(codes: np.ndarray, words: np.ndarray) -> np.ndarray:
    codes = np.ascontiguousarray(codes, np.uint16)
    nblk = (codes.size + N.SBM_BLOCK - 1) // N.SBM_BLOCK
    out = np.zeros(max(nblk, 1), np.uint32)
    check(lib().sbm_block_starts(codes.ctypes.data, codes.size,
                                 np.ascontiguousarray(words, np.uint32).ctypes.data, out.ctypes.data))
    return out[:nblk]


def validate_stream(codes, row_off, rows: int, cols: int, words) -> None:
    codes = np.ascontiguousarray(codes, np.uint16)
    row_off = np.ascontiguousarray(row_off, np.uint32)
    check(lib().sbm_validate_stream(codes.ctypes.data, codes.size, row_off.ctypes.data, rows, cols,
                                    np.ascontiguousarray(words, np.uint32).ctypes.data))

# ------------------------------------------------------------------ device data

@dataclass
class ExpertStack:
    """Encoded matrices of one shape (one projection of all experts), resident
    on the device in the layout the fused kernel reads."""
    rows: int
    cols: int
    n_experts: int
    codes: object      # torch.int16 [total codes] (uint16 bit patterns)
    row_off: object    # torch.int32 [E*(rows+1)] (uint32 values)
    bstart: object     # torch.int32 [total blocks]
    scales: object     # torch.float16 [E*rows]
    desc: object       # torch.uint8 [E*sizeof(MatrixDesc)]
    host_desc: list
    code_bytes: int    # bytes of codes actually used (without alignment padding)

    def matrix_bytes(self, e: int) -> int:
        """Bytes the fused kernel must read for expert e: codes + block starts
        + scales (row offsets are read once per slice)."""
        d = self.host_desc[e]
        nblk = (d.n_codes + N.SBM_BLOCK - 1) // N.SBM_BLOCK
        per_row = max(1, int(self.scales.numel()) // max(1, self.n_experts * self.rows))   # 1, or 2 (min/max)
        return 2 * d.n_codes + 4 * nblk + 2 * per_row * self.rows

    @staticmethod
    def from_symbols(syms, scales, words, device="cuda"):
        """Matrices of one shape (uint8 0/1/2) encoded by sbm_encode_experts and
        uploaded; scales: per matrix, rows fp16 (or [rows, 2] for the min/max
        grid, whose descriptors then get doubled scale bases)."""
        codes, row_off, bstart, descs = encode_experts(syms, words)
        rows, cols = syms[0].shape
        sc = [np.asarray(s, np.float16).reshape(-1) for s in scales]
        per_row = sc[0].size // rows
        assert all(s.size == per_row * rows for s in sc) and per_row in (1, 2)
        for d in descs:
            d.scale_base *= per_row
        used = 2 * sum(int(d.n_codes) for d in descs)
        return ExpertStack._upload(rows, cols, descs, codes, row_off, bstart, np.concatenate(sc), used, device)

    @staticmethod
    def _upload(rows, cols, descs, codes, row_off, bstart, scales, used, device):
        import torch
        if codes.size == 0:
            codes = np.zeros(8, np.uint16)
        if bstart.size == 0:
            bstart = np.zeros(1, np.uint32)
        desc_arr = (N.MatrixDesc * len(descs))(*descs)
        desc_bytes = np.frombuffer(bytes(desc_arr), np.uint8).copy()
        t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a).view(dt)).to(device)
        return ExpertStack(rows, cols, len(descs), t(codes, np.int16), t(row_off, np.int32),
                           t(bstart, np.int32), t(scales, np.float16), t(desc_bytes, np.uint8), descs, used)

    @staticmethod
    def assemble(mats, rows: int, cols: int, dict_tag: int):
        """Host stack layout from per-matrix encodings made with the dictionary
        whose tag is dict_tag (api.dict_tag(words)): (descs, codes, row_off,
        bstart, scales, used bytes)."""
        descs = []
        code_parts, off_parts, blk_parts, sc_parts = [], [], [], []
        cb = ob = sb = bb = 0
        used = 0
        for codes, row_off, bstart, scales in mats:
            n = int(codes.size)
            # one scale per row, or (w_min, w_max) per row for the min/max grid
            assert row_off.size == rows + 1 and scales.size in (rows, 2 * rows)
            d = N.MatrixDesc(code_base=cb, off_base=ob, scale_base=sb, blk_base=bb, n_codes=n,
                             rows=rows, cols=cols, dict_tag=dict_tag)
            descs.append(d)
            pad = (-n) % N.SBM_CODE_ALIGN
            code_parts.append(np.concatenate([codes.astype(np.uint16), np.zeros(pad, np.uint16)]))
            off_parts.append(row_off.astype(np.uint32))
            blk_parts.append(bstart.astype(np.uint32))
            sc_parts.append(scales.astype(np.float16))
            cb += n + pad
            ob += rows + 1
            sb += scales.size
            bb += bstart.size
            used += 2 * n
        codes = np.concatenate(code_parts) if code_parts else np.zeros(0, np.uint16)
        bstart = np.concatenate(blk_parts) if blk_parts else np.zeros(0, np.uint32)
        return descs, codes, np.concatenate(off_parts), bstart, np.concatenate(sc_parts), used

    @staticmethod
    def from_host(mats, rows: int, cols: int, device="cuda", *, dict_tag: int):
        """mats: list of (codes uint16, row_off uint32, bstart uint32, scales fp16),
        encoded with the dictionary whose tag is dict_tag (api.dict_tag(words))."""
        descs, codes, row_off, bstart, scales, used = ExpertStack.assemble(mats, rows, cols, dict_tag)
        return ExpertStack._upload(rows, cols, descs, codes, row_off, bstart, scales, used, device)


def device_image(words: np.ndarray, device="cuda", slots: int = 3):
    import torch
    return torch.from_numpy(dict_image(words, slots)).to(device)

# ------------------------------------------------------------------ GPU calls

def decode_ref(codes_t, row_off_t, rows: int, cols: int, words_t, stream=None, out=None, bad=None):
    """GPU reference decode of one matrix -> (symbols uint8 [rows, cols], bad_rows)."""
    import torch
    if out is None:
        out = _made_on(stream, torch.empty, (rows, cols), dtype=torch.uint8, device=codes_t.device)
    if bad is None:
        bad = _made_on(stream, torch.zeros, 1, dtype=torch.int32, device=codes_t.device)
    check(lib().sbm_decode_ref(_ptr(codes_t), _ptr(row_off_t), rows, cols, _ptr(words_t), _ptr(out),
                               _ptr(bad), _stream(stream)))
    return out, bad


def decode_dense(stack: "ExpertStack", e: int, image_t, out=None, bad=None, stream=None):
    """Expert e's matrix of a stack decoded to dense fp16 {-1, 0, +1}
    [rows, cols] (sbm_decode_dense; the row scales are not applied)."""
    import torch
    d = stack.host_desc[e]
    if out is None:
        out = _made_on(stream, torch.empty, (stack.rows, stack.cols), dtype=torch.float16, device=stack.codes.device)
    if bad is None:
        bad = _made_on(stream, torch.zeros, 1, dtype=torch.int32, device=stack.codes.device)
    check(lib().sbm_decode_dense(_ptr(stack.codes[d.code_base:]), int(d.n_codes), _ptr(stack.bstart[d.blk_base:]),
                                 stack.rows, stack.cols, _ptr(image_t), int(d.dict_tag), _ptr(out), _ptr(bad),
                                 _stream(stream)))
    return out, bad


def workspace_bytes(n_experts: int, n_tokens: int) -> int:
    return int(lib().sbm_workspace_bytes(n_experts, n_tokens))


def alloc_workspace(n_experts: int, n_tokens: int, device="cuda"):
    import torch
    return torch.empty(max(workspace_bytes(n_experts, n_tokens), 16), dtype=torch.uint8, device=device)


def _x_flag(x) -> int:
    """Activation dtype flag: fp16 (none) or bf16 (SBM_F_IN_BF16)."""
    import torch
    if x is None or x.dtype == torch.float16:
        return 0
    if x.dtype == torch.bfloat16:
        return N.SBM_F_IN_BF16
    raise TypeError(f"activations must be float16 or bfloat16, not {x.dtype}")


def moe_fused_decode_matvec(stack: ExpertStack, image_t, x, expert_ids, relu: bool = False,
                            out_f32: bool = False, workspace=None, y=None, stream=None, in_rms: bool = False,
                            mfma: bool = False, minmax: bool = False, image4=None,
                            deterministic: bool = False):
    """y[t] = act(W_{expert_ids[t]} x[t]) for one projection of an MoE layer
    (in_rms: x[t] is first scaled to unit RMS, as rms_glue does; mfma=True
    sends experts with 16 or more tokens to the dense-tile MFMA path; minmax:
    the stack's scales are (w_min, w_max) per row, the page's grid; image4:
    image_t is a 4-slot image, by default told from its byte size;
    deterministic: fixed-point row accumulators, bit-reproducible outputs)."""
    import torch
    T = int(x.shape[0]) if x is not None else 0
    if y is None:
        y = _made_on(stream, torch.empty, (T, stack.rows), dtype=torch.float32 if out_f32 else torch.float16,
                     device=stack.codes.device)
    if workspace is None:
        workspace = _made_on(stream, alloc_workspace, stack.n_experts, T, device=stack.codes.device)
    flags = (N.SBM_F_RELU if relu else 0) | (N.SBM_F_OUT_F32 if out_f32 else 0) | (N.SBM_F_IN_RMS if in_rms else 0)
    flags |= N.SBM_F_MFMA if mfma else 0
    flags |= N.SBM_F_MINMAX if minmax else 0
    flags |= N.SBM_F_DETERMINISTIC if deterministic else 0
    flags |= _x_flag(x)
    n4 = int(lib().sbm_dict_image4_bytes())
    if image4 is None:
        image4 = int(image_t.numel()) == n4
    need = n4 if image4 else int(lib().sbm_dict_image_bytes())
    if int(image_t.numel()) * image_t.element_size() < need:
        raise ValueError(f"image buffer holds {image_t.numel() * image_t.element_size()} bytes; the kernel copies {need}")
    flags |= N.SBM_F_IMAGE4 if image4 else 0
    check(lib().sbm_moe_fused_decode_matvec(
        _ptr(stack.codes), _ptr(stack.row_off), _ptr(stack.bstart), _ptr(stack.scales), _ptr(stack.desc),
        stack.n_experts, stack.rows, stack.cols, _ptr(image_t), _ptr(x), _ptr(expert_ids), T, _ptr(y),
        flags, _ptr(workspace), int(workspace.numel()), _stream(stream)))
    return y


def ffn_workspace_bytes(n_experts: int, n_tokens: int) -> int:
    return int(lib().sbm_ffn_workspace_bytes(n_experts, n_tokens))


def alloc_ffn_workspace(n_experts: int, n_tokens: int, device="cuda"):
    """Zeroed workspace of the layer call (it must start zeroed; every call
    leaves it ready for the next)."""
    import torch
    return torch.zeros(max(ffn_workspace_bytes(n_experts, n_tokens), 64), dtype=torch.uint8, device=device)


def _projection(st: ExpertStack):
    return N.Projection(codes=_ptr(st.codes), row_off=_ptr(st.row_off), bstart=_ptr(st.bstart),
                        scales=_ptr(st.scales), experts=_ptr(st.desc), n_experts=st.n_experts, rows=st.rows,
                        cols=st.cols)


def moe_fused_ffn(up: ExpertStack, down: ExpertStack, image_t, x, expert_ids, h=None, y=None, workspace=None,
                  in_rms: bool = False, out_f32: bool = False, stream=None):
    """One MoE expert FFN in one launch (sbm_moe_fused_ffn): h = relu(W_up x),
    y = W_down h for every token's expert.  Returns (y, h)."""
    import torch
    T = int(x.shape[0])
    dev = up.codes.device
    if h is None:
        h = _made_on(stream, torch.empty, (T, up.rows), dtype=torch.float16, device=dev)
    if y is None:
        y = _made_on(stream, torch.empty, (T, down.rows), dtype=torch.float32 if out_f32 else torch.float16, device=dev)
    if workspace is None:
        workspace = _made_on(stream, alloc_ffn_workspace, up.n_experts, T, dev)
    flags = (N.SBM_F_IN_RMS if in_rms else 0) | (N.SBM_F_OUT_F32 if out_f32 else 0) | _x_flag(x)
    pu, pd = _projection(up), _projection(down)
    check(lib().sbm_moe_fused_ffn(C.addressof(pu), C.addressof(pd), _ptr(image_t), _ptr(x), _ptr(expert_ids), T,
                                  _ptr(h), _ptr(y), flags, _ptr(workspace), int(workspace.numel()), _stream(stream)))
    return y, h


def layers_workspace_bytes(n_layers: int, n_experts: int, n_tokens: int) -> int:
    return int(lib().sbm_layers_workspace_bytes(n_layers, n_experts, n_tokens))


def alloc_layers_workspace(n_layers: int, n_experts: int, n_tokens: int, device="cuda"):
    """Zeroed workspace of the multi-layer call (it must start zeroed; every
    call leaves it ready for the next)."""
    import torch
    return torch.zeros(max(layers_workspace_bytes(n_layers, n_experts, n_tokens), 64), dtype=torch.uint8,
                       device=device)


def moe_fused_layers(ups, downs, image_t, x, expert_ids, h=None, y=None, workspace=None, in_rms: bool = False,
                     stream=None):
    """len(ups) MoE layers in one launch (sbm_moe_fused_layers): per layer l,
    h_l = relu(W_up x_l), y_l = W_down h_l with x_0 = x and x_l = y_{l-1}
    scaled to unit RMS per token; expert_ids: int32 [n_layers, T].  Returns
    (y, h): every layer's outputs, fp16 [n_layers, T, width]."""
    import torch
    L = len(ups)
    assert L == len(downs) and L >= 1
    T = int(x.shape[0])
    dev = ups[0].codes.device
    if h is None:
        h = _made_on(stream, torch.empty, (L, T, ups[0].rows), dtype=torch.float16, device=dev)
    if y is None:
        y = _made_on(stream, torch.empty, (L, T, downs[0].rows), dtype=torch.float16, device=dev)
    assert h.numel() >= L * T * ups[0].rows and y.numel() >= L * T * downs[0].rows
    if workspace is None:
        workspace = _made_on(stream, alloc_layers_workspace, L, ups[0].n_experts, T, dev)
    flags = (N.SBM_F_IN_RMS if in_rms else 0) | _x_flag(x)
    pu = (N.Projection * L)(*[_projection(u) for u in ups])
    pd = (N.Projection * L)(*[_projection(d) for d in downs])
    check(lib().sbm_moe_fused_layers(C.addressof(pu), C.addressof(pd), L, _ptr(image_t), _ptr(x), _ptr(expert_ids),
                                     T, _ptr(h), _ptr(y), flags, _ptr(workspace), int(workspace.numel()),
                                     _stream(stream)))
    return y, h


def workspace_error(workspace, stream=None) -> int:
    v = C.c_uint32()
    check(lib().sbm_workspace_error(_ptr(workspace), C.addressof(v), _stream(stream)))
    return int(v.value)

# ------------------------------------------------------------------ attention side

@dataclass
class KVCache:
    """Paged keys and values of one layer in 4 bits (the layout at "the
    attention's side" of include/sbm.h): data uint8 [n_blocks, n_kv_heads,
    block_size * head_dim * 17 / 16]."""
    data: object
    block_size: int
    head_dim: int

    @property
    def n_blocks(self) -> int:
        return int(self.data.shape[0])

    @property
    def n_kv_heads(self) -> int:
        return int(self.data.shape[1])


def alloc_kv_cache(n_blocks: int, n_kv_heads: int, head_dim: int, block_size: int = 16, device="cuda") -> KVCache:
    import torch
    if not int(lib().sbm_kv_cache_bytes(n_blocks, n_kv_heads, block_size, head_dim)):
        raise ValueError(f"no such cache: {n_blocks} blocks, {n_kv_heads} heads of {head_dim}, {block_size} tokens a block")
    return KVCache(torch.zeros(n_blocks, n_kv_heads, block_size * head_dim * 17 // 16, dtype=torch.uint8, device=device),
                   block_size, head_dim)


def rope_table(n_positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """fp32 [n_positions, rot_dim]: cosines, then sines, of position *
    base^(-2i / rot_dim), from angles in 64 bits."""
    import torch
    inv = torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(n_positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(device)


# What the calls below cost the host is what a decode step of few tokens costs, so a tensor's checks are one expression
# that looks at each property once; the slow path says which of them failed.
_pack_heads = struct.Struct("Pqq").pack            # sbm_heads: address, token stride, head stride


def _dev(t, what: str, dtype, at: int, contiguous: bool = True):
    """A device tensor's address; TypeError / ValueError where it cannot be what the kernels take.  at: the device's index."""
    if t.dtype is dtype and t.get_device() == at >= 0 and (not contiguous or t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    if t.get_device() != at:
        raise ValueError(f"{what} is on {t.device}, not the device of the others" + ("" if at < 0 else f" ({at})"))
    raise ValueError(f"{what} must be contiguous")


def _heads(t, what: str, dtype, at: int, shape):
    """[tokens, heads, head_dim] with any strides but the last as sbm_heads."""
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, head_dim] with neighbouring dimensions")
    ts, hs, ds = t.stride()
    if ds != 1 and t.shape[2] > 1:
        raise ValueError(f"{what} must be [tokens, heads, head_dim] with neighbouring dimensions")
    if t.shape != shape:
        raise ValueError(f"{what} is {tuple(t.shape)}, not {tuple(shape)}")
    return _pack_heads(_dev(t, what, dtype, at, False), ts, hs)


def _error(t, at: int):
    import torch
    if t is None:
        return 0
    if t.numel() < 1:
        raise ValueError("error must hold one int32")
    return _dev(t, "error", torch.int32, at)


@dataclass
class KVPlan:
    """What one serving step needs of its requests (sbm_kv_plan), all int32:
    slots, positions, requests [max_tokens]; cu_q [n_requests + 1]; kv_lens
    [n_requests]; n_free, error [1] (error collects: zero it to use it again);
    block_table [n_requests, width], the caller's, updated in place."""
    slots: object
    positions: object
    requests: object
    cu_q: object
    kv_lens: object
    n_free: object
    error: object
    block_table: object


_error_words = {}                                  # (device, stream) -> (zeroed int32 words, how many were given out)
_error_lock = threading.Lock()                     # threads share the default stream


def _error_word(at: int):
    """A zeroed int32 [1] that is given out once: filled 1024 at a time, on the stream that uses them."""
    import torch
    if torch.cuda.is_current_stream_capturing():   # the graph zeroes it at each replay
        return torch.zeros(1, dtype=torch.int32, device=f"cuda:{at}")
    key = at, _stream()
    with _error_lock:
        words, given = _error_words.get(key, (None, 1024))
        if given == 1024:
            words, given = torch.zeros(1024, dtype=torch.int32, device=f"cuda:{at}"), 0
        _error_words[key] = words, given + 1
    return words[given:given + 1]


def alloc_kv_plan(n_requests: int, max_tokens: int, block_table=None, device="cuda") -> KVPlan:
    """A plan to be filled (kv_plan); its error word is zero, the rest is not."""
    import torch
    n, r = max_tokens, n_requests
    on = torch.device(device) if block_table is None else block_table.device
    buf = torch.empty(3 * n + 2 * r + 2, dtype=torch.int32, device=on)
    at = buf.get_device()
    error = _error_word(at) if at >= 0 else torch.zeros(1, dtype=torch.int32)
    return KVPlan(*buf.split((n, n, n, r + 1, r, 1)), error, block_table)


def kv_plan(context_lens, new_lens, free_blocks, n_free, block_table, n_blocks: int, block_size: int, max_tokens: int,
            plan: KVPlan = None, stream=None) -> KVPlan:
    """Block tables and slot maps of one serving step from the requests' lengths
    (sbm_kv_plan): request i holds context_lens[i] tokens and gets new_lens[i];
    blocks it lacks are popped from the end of free_blocks[:n_free].  Nothing is
    read back: n_free and the error word stay on the device (plan.error:
    SBM_PLAN_E* bits, and then nothing was given out).  plan: one from
    alloc_kv_plan, to be filled again."""
    import torch
    i32 = torch.int32
    R = context_lens.numel()
    if new_lens.numel() != R or block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("context_lens, new_lens and block_table must have one row for each request")
    if n_free.numel() != 1:
        raise ValueError("n_free must hold one int32")
    at = context_lens.get_device()
    ins = (_dev(context_lens, "context_lens", i32, at), _dev(new_lens, "new_lens", i32, at), R,
           _dev(free_blocks, "free_blocks", i32, at), free_blocks.numel(), _dev(n_free, "n_free", i32, at),
           _dev(block_table, "block_table", i32, at))
    if plan is None:
        plan = alloc_kv_plan(R, max_tokens, block_table) if stream is None else \
            _made_on(stream, alloc_kv_plan, R, max_tokens, block_table)
        n = 4 * max_tokens
        p = plan.cu_q.data_ptr() - 3 * n           # one buffer, in this order
        outs = (p, p + n, p + 2 * n, p + 3 * n, p + 3 * n + 4 * R + 4, p + 3 * n + 8 * R + 4, plan.error.data_ptr())
    else:
        if plan.slots.numel() < max_tokens or plan.positions.numel() < max_tokens or plan.requests.numel() < max_tokens \
                or plan.cu_q.numel() < R + 1 or plan.kv_lens.numel() < R:
            raise ValueError("the plan was made for fewer requests or tokens")
        plan.block_table = block_table
        outs = (_dev(plan.slots, "slots", i32, at), _dev(plan.positions, "positions", i32, at),
                _dev(plan.requests, "requests", i32, at), _dev(plan.cu_q, "cu_q", i32, at),
                _dev(plan.kv_lens, "kv_lens", i32, at), _dev(plan.n_free, "plan.n_free", i32, at), _error(plan.error, at))
    check(lib().sbm_kv_plan(*ins, block_table.shape[1], n_blocks, block_size, max_tokens, *outs, _stream(stream, at)))
    return plan


def _qk_norm_rope(q, k, v, q_weight, k_weight, positions, rope, eps, neighbours, q_out, k_out, slots, cache, error,
                  stream):
    import torch
    dtype, at, shape = q.dtype, q.get_device(), q.shape
    flags = _x_flag(q) | (N.SBM_F_NEIGHBOURS if neighbours else 0)
    hq = _heads(q, "q", dtype, at, shape)
    T, H, D = shape
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, head_dim]")
    Hk = k.shape[1]
    kshape = (T, Hk, D)
    hk = _heads(k, "k", dtype, at, kshape)
    hv = None if v is None else _heads(v, "v", dtype, at, kshape)
    wq = wk = pos = rp = rows = rot = 0
    if q_weight is not None:
        if q_weight.numel() != D:
            raise ValueError(f"q_weight must hold {D} elements")
        wq = _dev(q_weight, "q_weight", dtype, at)
    if k_weight is not None:
        if k_weight.numel() != D:
            raise ValueError(f"k_weight must hold {D} elements")
        wk = _dev(k_weight, "k_weight", dtype, at)
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [positions, rot_dim]")
        rows, rot = rope.shape
        rp = _dev(rope, "rope", torch.float32, at)
        if positions is None or positions.numel() != T:
            raise ValueError(f"positions must hold {T} elements")
        pos = _dev(positions, "positions", torch.int32, at)
    if q_out is None:
        q_out = q.new_empty(shape) if stream is None else _made_on(stream, q.new_empty, shape)
        ho = _pack_heads(q_out.data_ptr(), H * D, D)
    else:
        ho = _heads(q_out, "q_out", dtype, at, shape)
    if k_out is None and cache is None:
        k_out = q.new_empty(kshape) if stream is None else _made_on(stream, q.new_empty, kshape)
        hko = _pack_heads(k_out.data_ptr(), Hk * D, D)
    else:
        hko = None if k_out is None else _heads(k_out, "k_out", dtype, at, kshape)
    sl = data = nb = bs = 0
    if cache is not None:
        data, nb, hc = _cache(cache, at)
        if hc != Hk or cache.head_dim != D:
            raise ValueError(f"the cache holds {hc} heads of {cache.head_dim}, not {Hk} of {D}")
        if v is None:
            raise ValueError("v must be given with a cache")
        sl, bs = _slots(slots, T, at), cache.block_size
    check(lib().sbm_qk_norm_rope(hq, hk, hv, wq, wk, pos, rp, rows, rot, eps, T, H, Hk, D, ho, hko, sl, data, nb, bs, flags,
                                 _error(error, at), _stream(stream, at)))
    return q_out, k_out


def _slots(slots, n: int, at: int):
    import torch
    if slots is None or slots.numel() != n:
        raise ValueError(f"slots must hold {n} elements")
    return _dev(slots, "slots", torch.int32, at)


def _cache(cache: KVCache, at: int):
    """(address, blocks, key heads)"""
    import torch
    d = cache.data
    if d.dim() != 3 or d.shape[2] != cache.block_size * cache.head_dim * 17 // 16:
        raise ValueError(f"a cache of {tuple(d.shape)} bytes holds no blocks of {cache.block_size} x {cache.head_dim}")
    return _dev(d, "cache", torch.uint8, at), d.shape[0], d.shape[1]


def qk_norm_rope(q, k, q_weight, k_weight, positions, rope, eps: float = 1e-6, neighbours: bool = False, q_out=None,
                 k_out=None, error=None, stream=None):
    """Norm of each head of q [T, heads, D] and k [T, kv_heads, D] by its weight
    [D] (None: ones) and rotation by rope[positions[t]] (rope_table; None: no
    rotation; neighbours: pairs (2i, 2i + 1) instead of halves), in one launch
    (sbm_qk_norm_rope).  Returns (q_out, k_out); they may be q and k."""
    return _qk_norm_rope(q, k, None, q_weight, k_weight, positions, rope, eps, neighbours, q_out, k_out, None, None, error,
                         stream)


def qk_norm_rope_store(q, k, v, q_weight, k_weight, positions, rope, slots, cache: KVCache, eps: float = 1e-6,
                       neighbours: bool = False, q_out=None, k_out=None, error=None, stream=None):
    """qk_norm_rope whose keys go, with the values v, into the 4-bit cache at
    slots[t] (negative: nowhere) in the same launch; k_out: the keys too.
    Returns q_out."""
    return _qk_norm_rope(q, k, v, q_weight, k_weight, positions, rope, eps, neighbours, q_out, k_out, slots, cache, error,
                         stream)[0]


def kv_load(cache: KVCache, slots, dtype=None, k=None, v=None, error=None, stream=None):
    """The cached tokens at slots as values (sbm_kv_load): k, v [n, kv_heads, D]
    in float16 (or bfloat16); a negative slot gives zeros."""
    import torch
    dtype = dtype or (torch.float16 if k is None else k.dtype)
    n, at = slots.numel(), slots.get_device()
    data, nb, Hk = _cache(cache, at)
    shape = (n, Hk, cache.head_dim)
    if k is None:
        k = slots.new_empty(shape, dtype=dtype) if stream is None else _made_on(stream, slots.new_empty, shape, dtype=dtype)
    if v is None:
        v = slots.new_empty(shape, dtype=dtype) if stream is None else _made_on(stream, slots.new_empty, shape, dtype=dtype)
    if k.shape != shape or v.shape != shape:
        raise ValueError(f"k and v must be {shape}, not {tuple(k.shape)} and {tuple(v.shape)}")
    check(lib().sbm_kv_load(data, nb, Hk, cache.block_size, cache.head_dim, _slots(slots, n, at), n, _dev(k, "k", dtype, at),
                            _dev(v, "v", dtype, at), _x_flag(k), _error(error, at), _stream(stream, at)))
    return k, v


def attention_workspace_bytes(n_requests: int, n_tokens: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(lib().sbm_attention_kv4_workspace_bytes(n_requests, n_tokens, n_heads, n_kv_heads, head_dim))


def alloc_attention_workspace(n_requests: int, n_tokens: int, n_heads: int, n_kv_heads: int, head_dim: int,
                              device="cuda"):
    """Workspace of the attention, its head zeroed (it must start so; every call
    leaves it ready for the next)."""
    import torch
    n = max(attention_workspace_bytes(n_requests, n_tokens, n_heads, n_kv_heads, head_dim), N.SBM_ATTENTION_ZEROED)
    t = torch.empty(n, dtype=torch.uint8, device=device)
    t[:N.SBM_ATTENTION_ZEROED].zero_()
    return t


def attention_kv4(q, cache: KVCache, block_table, kv_lens, cu_q=None, scale: float = None, out=None, lse=None,
                  return_lse: bool = False, workspace=None, error=None, stream=None):
    """Attention of each request's last tokens over its cached ones
    (sbm_attention_kv4): q [T, heads, D], of request r the rows cu_q[r] ..
    cu_q[r + 1] (cu_q None: one token each), which see the request's kv_lens[r]
    tokens up to their own.  scale: 1 / sqrt(D) by default.  Returns out [T,
    heads, D], or (out, lse fp32 [T, heads]) with return_lse or an lse buffer."""
    import torch
    i32 = torch.int32
    dtype, at, shape = q.dtype, q.get_device(), q.shape
    if len(shape) != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    T, H, D = shape
    R = kv_lens.numel()
    Hk = cache.n_kv_heads
    if cache.head_dim != D or H % Hk:
        raise ValueError(f"the cache holds {Hk} heads of {cache.head_dim}; q has {H} of {D}")
    if block_table.dim() != 2 or block_table.shape[0] != R or (cu_q is not None and cu_q.numel() != R + 1):
        raise ValueError("kv_lens, block_table and cu_q must be of the same requests")
    hq = _heads(q, "q", dtype, at, shape)
    data, nb, _ = _cache(cache, at)
    if out is None:
        out = q.new_empty(shape) if stream is None else _made_on(stream, q.new_empty, shape)
        po = out.data_ptr()
    elif out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, not {tuple(out.shape)}")
    else:
        po = _dev(out, "out", dtype, at)
    pl = 0
    if lse is not None:
        if lse.shape != (T, H):
            raise ValueError(f"lse must be {(T, H)}, not {tuple(lse.shape)}")
        pl = _dev(lse, "lse", torch.float32, at)
    elif return_lse:
        lse = q.new_empty((T, H), dtype=torch.float32) if stream is None else \
            _made_on(stream, q.new_empty, (T, H), dtype=torch.float32)
        pl = lse.data_ptr()
    if workspace is None:
        workspace = _made_on(stream, alloc_attention_workspace, R, T, H, Hk, D, q.device)
    check(lib().sbm_attention_kv4(
        hq, data, nb, cache.block_size, _dev(block_table, "block_table", i32, at), block_table.shape[1],
        _dev(kv_lens, "kv_lens", i32, at), 0 if cu_q is None else _dev(cu_q, "cu_q", i32, at), R, T, H, Hk, D,
        D ** -0.5 if scale is None else scale, po, pl, _x_flag(q), _dev(workspace, "workspace", torch.uint8, at),
        workspace.numel(), _error(error, at), _stream(stream, at)))
    return out if lse is None else (out, lse)

# ------------------------------------------------------------------ synthetic stacks

def build_trie(words: np.ndarray) -> np.ndarray:
    """Host trie child table (int32[(65536+1)*9]) of a dictionary."""
    out = np.zeros(int(lib().sbm_trie_words()), np.int32)
    check(lib().sbm_build_trie(np.ascontiguousarray(words, np.uint32).ctypes.data, out.ctypes.data))
    return out


def generate_stack(seed: int, layer: int, n_experts: int, mat: int, rows: int, cols: int, p0: float,
                   trie_t, scale_table_t, stream=None, *, dict_checksum: int) -> ExpertStack:
    """Generate and encode n_experts counter-based matrices on the GPU
    (count pass, row offsets, descriptors, write pass) as an ExpertStack;
    dict_checksum: the checksum of the dictionary the trie was built from."""
    import torch
    from . import synth
    if stream is not None:                             # sizes are read back and buffers made between the passes
        with torch.cuda.stream(stream):
            return generate_stack(seed, layer, n_experts, mat, rows, cols, p0, trie_t, scale_table_t,
                                  dict_checksum=dict_checksum)
    dev = trie_t.device
    z = synth.zero_threshold16(p0)
    s = _stream()
    counts = torch.empty(n_experts * rows, dtype=torch.int32, device=dev)
    check(lib().sbm_gen_count(seed, layer, n_experts, mat, rows, cols, z, _ptr(trie_t), _ptr(counts), s))
    row_off = torch.empty(n_experts * (rows + 1), dtype=torch.int32, device=dev)
    desc = torch.empty(n_experts * C.sizeof(N.MatrixDesc), dtype=torch.uint8, device=dev)
    totals = torch.zeros(2, dtype=torch.int64, device=dev)
    check(lib().sbm_gen_layout(_ptr(counts), n_experts, rows, cols, _ptr(row_off), _ptr(desc), _ptr(totals),
                               C.c_uint64(dict_checksum), s))
    tot = totals.cpu().tolist()
    codes = torch.empty(max(int(tot[0]), 8), dtype=torch.int16, device=dev)
    bstart = torch.empty(max(int(tot[1]), 1), dtype=torch.int32, device=dev)
    scales = torch.empty(n_experts * rows, dtype=torch.float16, device=dev)
    check(lib().sbm_gen_write(seed, layer, n_experts, mat, rows, cols, z, _ptr(trie_t), _ptr(row_off),
                              _ptr(desc), _ptr(codes), _ptr(bstart), _ptr(scale_table_t), _ptr(scales), s))
    del counts
    host_desc = list((N.MatrixDesc * n_experts).from_buffer_copy(desc.cpu().numpy().tobytes()))
    used = 2 * sum(int(d.n_codes) for d in host_desc)
    return ExpertStack(rows, cols, n_experts, codes, row_off, bstart, scales, desc, host_desc, used)


def stream_read(buf, sink, stream=None) -> None:
    """Bandwidth probe: read every byte of the device tensor buf (sbm_stream_read)."""
    check(lib().sbm_stream_read(_ptr(buf), int(buf.numel() * buf.element_size()), _ptr(sink), int(sink.numel()),
                                _stream(stream)))


def rms_glue(y, out=None, stream=None):
    """Stack glue (not the method): x_next = y / rms(y) per token, fp16."""
    import torch
    if out is None:
        out = _made_on(stream, torch.empty_like, y)
    check(lib().sbm_rms_glue(_ptr(y), int(y.shape[0]), int(y.shape[1]), _ptr(out), _stream(stream)))
    return out
