"""ctypes marshalling for libpkv.so (argument checks and pointers only)."""
import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG, "libpkv.so")
_lib = None

DEV_ERR_BITS = {
    "SLOT_RANGE": 1,
    "QSL": 2,
    "SEQ_LEN": 4,
    "BT_WIDTH": 8,
    "BLOCK_ID": 16,
    "TIMEOUT": 32,
    "INT8_PREFILL": 64,
    "CAPACITY": 128,
    "POSITION": 256,
}

EXPORTS = ["pkv_write", "pkv_attention", "pkv_reserve_workspace", "pkv_get_error",
           "pkv_last_error_string", "pkv_num_sms", "pkv_trace_enable", "pkv_trace_read",
           "pkv_launch_count", "pkv_prepare_step", "pkv_write_int8", "pkv_attention_int8",
           "pkv_plan", "pkv_attention_planned", "pkv_workspace_size", "pkv_write_rope",
           "pkv_write_rope_int8", "pkv_attention_scored", "pkv_write_rope_packed",
           "pkv_attention_scored_packed", "pkv_write_int4", "pkv_read_int4",
           "pkv_attention_int4", "pkv_page_bounds", "pkv_select_pages", "pkv_reserve_select",
           "pkv_attention_selected"]
INT4_PAGE_BYTES = 2176  # PKV_INT4_PAGE_BYTES of include/pkv.h
TRACE_KINDS = ["write", "plan", "decode", "prefill", "combine", "prepare"]


class PkvError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("pkv error %d: %s" % (code, msg))
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def load():
    """Loads libpkv.so (built by ``build.py`` / ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise PkvError(-100, "libpkv.so is not built (%s); run __graft_entry__.build()" % _LIB_PATH)
    L = ctypes.CDLL(_LIB_PATH)
    i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
    L.pkv_write.restype = ctypes.c_int
    L.pkv_write.argtypes = [vp, i64, vp, i64, vp, vp, i64, i32, i32, i32, vp, i64, vp]
    L.pkv_attention.restype = ctypes.c_int
    L.pkv_attention.argtypes = [vp, i64, i64, i32, vp, vp, i64, i32, i32, i32, vp, vp, vp, i64,
                                i32, f32, vp, i64, vp]
    f32 = ctypes.c_float
    L.pkv_attention_scored.restype = ctypes.c_int
    L.pkv_attention_scored.argtypes = [vp, i64, i64, i32, vp, vp, i64, i32, i32, i32, vp, vp, vp,
                                       i64, i32, f32, f32, i32, vp, vp, vp, i64, vp]
    L.pkv_write_rope_packed.restype = ctypes.c_int
    L.pkv_write_rope_packed.argtypes = [ctypes.c_char_p, ctypes.c_int]
    L.pkv_attention_scored_packed.restype = ctypes.c_int
    L.pkv_attention_scored_packed.argtypes = [ctypes.c_char_p]
    L.pkv_write_int8.restype = ctypes.c_int
    L.pkv_write_int8.argtypes = [vp, i64, vp, i64, vp, vp, f32, f32, i64, i32, i32, i32, vp, i64,
                                 vp]
    L.pkv_attention_int8.restype = ctypes.c_int
    L.pkv_attention_int8.argtypes = [vp, i64, i64, i32, vp, vp, f32, f32, i64, i32, i32, i32, vp,
                                     vp, vp, i64, i32, f32, vp, i64, vp]
    rope = [vp, i64, i32, vp, i64, vp, i64, vp, vp, f32, f32, vp, i64, i32, i32, vp, vp, i64, vp,
            vp]
    L.pkv_write_rope.restype = ctypes.c_int
    L.pkv_write_rope.argtypes = rope + [i64, i32, i32, i32, vp, i64, vp]
    L.pkv_write_rope_int8.restype = ctypes.c_int
    L.pkv_write_rope_int8.argtypes = rope + [f32, f32, i64, i32, i32, i32, vp, i64, vp]
    L.pkv_write_int4.restype = ctypes.c_int
    L.pkv_write_int4.argtypes = [vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, i64, vp]
    L.pkv_read_int4.restype = ctypes.c_int
    L.pkv_read_int4.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp]
    L.pkv_attention_int4.restype = ctypes.c_int
    L.pkv_attention_int4.argtypes = [vp, i64, i64, i32, vp, i64, i32, i32, i32, vp, vp, vp, i64,
                                     i32, f32, vp, i64, vp]
    L.pkv_page_bounds.restype = ctypes.c_int
    L.pkv_page_bounds.argtypes = [vp, i64, i32, i32, i32, vp, vp, i64, vp]
    L.pkv_select_pages.restype = ctypes.c_int
    L.pkv_select_pages.argtypes = [vp, i64, i64, i32, vp, i64, i32, i32, i32, vp, vp, vp, i64, i32,
                                   i32, i32, i32, vp, vp, vp]
    L.pkv_reserve_select.restype = ctypes.c_int
    L.pkv_reserve_select.argtypes = [i64, i64, i32]
    L.pkv_attention_selected.restype = ctypes.c_int
    L.pkv_attention_selected.argtypes = [vp, i64, i64, i32, vp, vp, i64, i32, i32, i32, vp, i64,
                                         vp, f32, vp, i64, vp]
    L.pkv_plan.restype = ctypes.c_int
    L.pkv_plan.argtypes = [i64, i32, i32, vp, vp, i64, i32, vp]
    L.pkv_attention_planned.restype = ctypes.c_int
    L.pkv_attention_planned.argtypes = [vp, i64, i32, vp, vp, i64, i32, i32, i32, vp, f32, vp,
                                        i64, vp]
    L.pkv_reserve_workspace.restype = ctypes.c_int
    L.pkv_reserve_workspace.argtypes = [i32, i64, i64, i32, i32]
    L.pkv_get_error.restype = ctypes.c_int
    L.pkv_get_error.argtypes = [vp, ctypes.POINTER(i32)]
    L.pkv_last_error_string.restype = ctypes.c_char_p
    L.pkv_last_error_string.argtypes = []
    L.pkv_num_sms.restype = ctypes.c_int
    L.pkv_num_sms.argtypes = []
    L.pkv_trace_enable.restype = ctypes.c_int
    L.pkv_trace_enable.argtypes = [ctypes.c_int]
    L.pkv_trace_read.restype = ctypes.c_int
    L.pkv_trace_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64),
                                 ctypes.c_int]
    L.pkv_launch_count.restype = i64
    L.pkv_launch_count.argtypes = []
    _lib = L
    return L


def _check(rc):
    if rc != 0:
        msg = load().pkv_last_error_string().decode(errors="replace")
        raise PkvError(rc, msg)


_torch = None
_raw_stream = None  # () -> the current device's current stream handle, as an int
_get_device = None  # () -> the current device's index


def _T():
    """torch, imported on first use (the binding loads without it)."""
    global _torch, _raw_stream, _get_device
    if _torch is None:
        import torch
        get_dev = getattr(torch._C, "_cuda_getDevice", None)
        get_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if get_dev is not None and get_raw is not None:
            _raw_stream = lambda: get_raw(get_dev())  # noqa: E731
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        # (a build or machine without CUDA has no current device, and no tensor on one)
        _get_device = torch.cuda.current_device
        if not torch.cuda.is_available():
            _get_device = lambda: -2  # noqa: E731
        elif get_dev is not None:
            _get_device = get_dev
        _torch = torch
    return _torch


def _stream(stream):
    """The stream handle for a call: torch's current stream when none is given
    (read through torch's raw getter: a Stream object costs microseconds)."""
    if stream is None:
        if _raw_stream is None:
            _T()
        return _raw_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _require(t, dtype, name, device=True):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)


def _per_row(t):
    """Elements in one row of a [rows, ...] tensor (also when it has no rows)."""
    n = 1
    for x in t.shape[1:]:
        n *= x
    return n


def _rows3(t, name):
    """Row stride of a [rows, heads, 128] tensor whose per-row block is contiguous
    (of one head or one row, that dimension's stride addresses nothing)."""
    st, sh = t.stride(), t.shape
    if len(st) == 2:
        if st[1] != 1:
            raise ValueError("%s: last dimension must be contiguous" % name)
    elif len(st) != 3 or st[2] != 1 or (st[1] != sh[2] and sh[1] != 1):
        raise ValueError("%s must be [rows, heads, head_size] with contiguous rows" % name)
    return _per_row(t) if sh[0] == 1 else st[0]


def _all_on_device(dtype, *ts):
    """True when every tensor has this dtype and lives on a CUDA device (the
    common case, tested in one pass; callers fall back to the per-argument
    checks, which name the culprit, when it is False)."""
    try:
        for t in ts:
            if t.dtype is not dtype or not t.is_cuda:
                return False
    except AttributeError:
        return False
    return True


def pkv_write(k, v, key_cache, value_cache, slot_mapping, n_tokens=None, stream=None):
    """Scatters k/v ([n, Hkv, 128] bf16) into the caches at slot_mapping (int64)."""
    torch = _T()
    if not (_all_on_device(torch.bfloat16, k, v, key_cache, value_cache) and
            _all_on_device(torch.int64, slot_mapping)):
        for t, n in ((k, "k"), (v, "v"), (key_cache, "key_cache"), (value_cache, "value_cache")):
            _require(t, torch.bfloat16, n)
        _require(slot_mapping, torch.int64, "slot_mapping")
    ks = key_cache.shape
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()) or len(ks) != 4:
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, head_size]")
    if ks != value_cache.shape:
        raise ValueError("key_cache and value_cache shapes differ")
    if not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous")
    nb, bs, hkv, d = ks
    n = slot_mapping.shape[0] if n_tokens is None else int(n_tokens)
    if n > slot_mapping.shape[0] or n > k.shape[0] or n > v.shape[0]:
        raise ValueError("n_tokens exceeds the rows of k/v/slot_mapping")
    _check(load().pkv_write(k.data_ptr(), _rows3(k, "k"), v.data_ptr(), _rows3(v, "v"),
                            key_cache.data_ptr(), value_cache.data_ptr(), nb, bs, hkv, d,
                            slot_mapping.data_ptr(), n, _stream(stream)))


def pkv_attention(q, key_cache, value_cache, query_start_loc, seq_lens, block_table, num_reqs,
                  scale, out, stream=None):
    """Causal varlen attention of q ([T, Hq, 128] bf16) over the paged cache
    into out ([T, Hq, 128] bf16); see include/pkv.h for the contract."""
    torch = _T()
    metadata = ((query_start_loc, "query_start_loc"), (seq_lens, "seq_lens"),
                (block_table, "block_table"))
    if not (_all_on_device(torch.bfloat16, q, key_cache, value_cache, out) and
            _all_on_device(torch.int32, query_start_loc, seq_lens, block_table)):
        for t, n in ((q, "q"), (key_cache, "key_cache"), (value_cache, "value_cache"),
                     (out, "out")):
            _require(t, torch.bfloat16, n)
        for t, n in metadata:
            _require(t, torch.int32, n)
    for t, n in metadata:
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    ks = key_cache.shape
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()) or len(ks) != 4:
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, head_size]")
    if ks != value_cache.shape:
        raise ValueError("key_cache and value_cache shapes differ")
    nb, bs, hkv, d = ks
    qs = q.shape
    if len(qs) != 3:
        raise ValueError("q must be [rows, num_heads, head_size]")
    rows, hq, _ = qs
    if out.shape[0] < rows or _per_row(out) != hq * d:
        raise ValueError("out must hold [rows, num_heads * head_size]")
    bts = block_table.shape
    bt_width = bts[1] if len(bts) == 2 else bts[0]
    num_reqs = int(num_reqs)
    if num_reqs > 0 and (query_start_loc.numel() < num_reqs + 1 or
                         seq_lens.numel() < num_reqs or
                         (len(bts) == 2 and bts[0] < num_reqs)):
        raise ValueError("metadata shorter than num_reqs")
    _check(load().pkv_attention(q.data_ptr(), _rows3(q, "q"), rows, hq, key_cache.data_ptr(),
                                value_cache.data_ptr(), nb, bs, hkv, d,
                                query_start_loc.data_ptr(), seq_lens.data_ptr(),
                                block_table.data_ptr(), bt_width, num_reqs, float(scale),
                                out.data_ptr(), _rows3(out, "out"), _stream(stream)))


def _caches(key_cache, value_cache, dtype):
    import torch
    for t, n in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        _require(t, dtype, n)
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()) or key_cache.dim() != 4:
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, head_size]")
    if key_cache.shape != value_cache.shape:
        raise ValueError("key_cache and value_cache shapes differ")
    return key_cache.shape


# The structs of the packed calls (pkv_write_rope_args, pkv_attention_scored_args
# of include/pkv.h): packed by one call and passed as one argument, they cost
# 0.5 us where two dozen ctypes arguments cost 2.2.
_ROPE_ARGS = struct.Struct("=19q6i4f")
_SCORED_ARGS = struct.Struct("=15q6i2f")


def _name_culprit(*named):
    """Raises for the first of these (tensor, name, dtype) triples that is no
    tensor of that dtype on the current CUDA device, whose stream the call
    enqueues on (None stands for an optional tensor left out)."""
    dev = _get_device()
    for t, name, dtype in named:
        if t is None:
            continue
        _require(t, dtype, name)
        if t.get_device() != dev:
            raise ValueError("%s is on cuda:%d, the current device is cuda:%d" %
                             (name, t.get_device(), dev))


def _write_rope(q, k, v, positions, cos_sin, key_cache, value_cache, slot_mapping, q_out,
                interleaved, q_weight, k_weight, weight_offset, eps, n_tokens, stream, scales):
    torch = _torch or _T()
    bf16 = torch.bfloat16
    cache = torch.int8 if scales else bf16
    # every check in one pass of plain attribute reads (a small step's time is
    # this function's); a failing one is named afterwards
    try:
        dev = _get_device()
        good = (q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16 and q_out.dtype is bf16 and
                key_cache.dtype is cache and value_cache.dtype is cache and
                cos_sin.dtype is torch.float32 and positions.dtype is torch.int64 and
                slot_mapping.dtype is torch.int64 and
                dev == q.get_device() == k.get_device() == v.get_device() == q_out.get_device() ==
                key_cache.get_device() == value_cache.get_device() == cos_sin.get_device() ==
                positions.get_device() == slot_mapping.get_device())
        qw = kw = 0
        if q_weight is not None:
            good = good and q_weight.dtype is bf16 and dev == q_weight.get_device()
            qw = q_weight.data_ptr()
        if k_weight is not None:
            good = good and k_weight.dtype is bf16 and dev == k_weight.get_device()
            kw = k_weight.data_ptr()
    except AttributeError:
        good = False
    if not good:
        _name_culprit((q, "q", bf16), (k, "k", bf16), (v, "v", bf16), (q_out, "q_out", bf16),
                      (key_cache, "key_cache", cache), (value_cache, "value_cache", cache),
                      (cos_sin, "cos_sin", torch.float32), (positions, "positions", torch.int64),
                      (slot_mapping, "slot_mapping", torch.int64), (q_weight, "q_weight", bf16),
                      (k_weight, "k_weight", bf16))
        raise ValueError("arguments must be tensors on the current CUDA device")
    cs = key_cache.shape
    if len(cs) != 4 or cs != value_cache.shape or not (key_cache.is_contiguous() and
                                                       value_cache.is_contiguous()):
        _caches(key_cache, value_cache, cache)
    nb, bs, hkv, d = cs
    try:
        rows, hq, qd = q.shape
        orows, ohq, od = q_out.shape
        krows, hk, kd = k.shape
        vrows, hv, vd = v.shape
        qs, q1, q2 = q.stride()
        os_, o1, o2 = q_out.stride()
        ks, k1, k2 = k.stride()
        vs, v1, v2 = v.stride()
        far, rot = cos_sin.shape
        n, = slot_mapping.shape
        npos, = positions.shape
    except ValueError:
        raise ValueError("q, k, v and q_out must be [rows, heads, head_size], cos_sin "
                         "[max_positions, rotary_dim], positions and slot_mapping "
                         "one-dimensional") from None
    if not (qd == od == kd == vd == d and ohq == hq and hk == hv == hkv):
        raise ValueError("q and q_out must have the same heads, k and v those of the caches, all "
                         "head_size %d" % d)
    if not (q2 == o2 == k2 == v2 == 1 and (q1 == o1 == d or hq == 1) and
            (k1 == v1 == d or hkv == 1)):
        raise ValueError("q, k, v and q_out must have contiguous rows")
    if not (cos_sin.is_contiguous() and slot_mapping.is_contiguous() and
            positions.is_contiguous()):
        raise ValueError("cos_sin, slot_mapping and positions must be contiguous")
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None and (t.shape != (d,) or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous [head_size]" % name)
    if n_tokens is not None:
        if int(n_tokens) > n:
            raise ValueError("n_tokens exceeds the rows of slot_mapping")
        n = int(n_tokens)
    if n > rows or n > orows or n > krows or n > vrows or n > npos:
        raise ValueError("n_tokens exceeds the rows of q/k/v/q_out/positions")
    if n == 1:  # (a single row's stride may be anything)
        qs = os_ = hq * d
        ks = vs = hkv * d
    try:
        args = _ROPE_ARGS.pack(
            q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, qw, kw, cos_sin.data_ptr(), far,
            positions.data_ptr(), q_out.data_ptr(), os_, key_cache.data_ptr(),
            value_cache.data_ptr(), nb, slot_mapping.data_ptr(), n,
            _raw_stream() if stream is None else _stream(stream), hq, hkv, d, bs, rot,
            1 if interleaved else 0, weight_offset, eps, *(scales or (0.0, 0.0)))
    except (struct.error, OverflowError) as e:
        raise ValueError("an argument is out of range: %s" % e) from None
    rc = (_lib or load()).pkv_write_rope_packed(args, 1 if scales else 0)
    if rc:
        _check(rc)


def pkv_write_rope(q, k, v, positions, cos_sin, key_cache, value_cache, slot_mapping, q_out,
                   interleaved=False, q_weight=None, k_weight=None, weight_offset=0.0, eps=1e-6,
                   n_tokens=None, stream=None):
    """pkv_write with the rotation of q and k ([n, heads, 128] bf16) at
    positions (int64) by cos_sin ([max_positions, rotary_dim] fp32, cos | sin),
    after a per-head RMS norm where a weight ([128] bf16) is given: rotated
    queries into q_out (q itself for in place), keys and values into the caches."""
    _write_rope(q, k, v, positions, cos_sin, key_cache, value_cache, slot_mapping, q_out,
                interleaved, q_weight, k_weight, weight_offset, eps, n_tokens, stream, ())


def pkv_write_rope_int8(q, k, v, positions, cos_sin, key_cache, value_cache, slot_mapping,
                        k_scale, v_scale, q_out, interleaved=False, q_weight=None, k_weight=None,
                        weight_offset=0.0, eps=1e-6, n_tokens=None, stream=None):
    """pkv_write_rope into int8 caches: codes clamp(rne(x / scale), -127, 127)
    of the rotated fp32 keys and of the values."""
    _write_rope(q, k, v, positions, cos_sin, key_cache, value_cache, slot_mapping, q_out,
                interleaved, q_weight, k_weight, weight_offset, eps, n_tokens, stream,
                (k_scale, v_scale))


def pkv_write_int8(k, v, key_cache, value_cache, slot_mapping, k_scale, v_scale, n_tokens=None,
                   stream=None):
    """Quantises k/v ([n, Hkv, 128] bf16) into the int8 caches at slot_mapping:
    code = clamp(rne(x / scale), -127, 127), one fp32 scale per cache."""
    import torch
    _require(k, torch.bfloat16, "k")
    _require(v, torch.bfloat16, "v")
    nb, bs, hkv, d = _caches(key_cache, value_cache, torch.int8)
    _require(slot_mapping, torch.int64, "slot_mapping")
    if not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous")
    n = slot_mapping.shape[0] if n_tokens is None else int(n_tokens)
    if n > slot_mapping.shape[0] or n > k.shape[0] or n > v.shape[0]:
        raise ValueError("n_tokens exceeds the rows of k/v/slot_mapping")
    _check(load().pkv_write_int8(k.data_ptr(), _rows3(k, "k"), v.data_ptr(), _rows3(v, "v"),
                                 key_cache.data_ptr(), value_cache.data_ptr(), float(k_scale),
                                 float(v_scale), nb, bs, hkv, d, slot_mapping.data_ptr(), n,
                                 _stream(stream)))


def pkv_attention_int8(q, key_cache, value_cache, k_scale, v_scale, query_start_loc, seq_lens,
                       block_table, num_reqs, scale, out, stream=None):
    """pkv_attention over int8 caches (K = code * k_scale, V = code * v_scale),
    decode-path requests only; see include/pkv.h."""
    import torch
    _require(q, torch.bfloat16, "q")
    _require(out, torch.bfloat16, "out")
    nb, bs, hkv, d = _caches(key_cache, value_cache, torch.int8)
    for t, n in ((query_start_loc, "query_start_loc"), (seq_lens, "seq_lens"),
                 (block_table, "block_table")):
        _require(t, torch.int32, n)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    if q.dim() != 3:
        raise ValueError("q must be [rows, num_heads, head_size]")
    rows, hq, _ = q.shape
    if out.shape[0] < rows or _per_row(out) != hq * d:
        raise ValueError("out must hold [rows, num_heads * head_size]")
    bt_width = block_table.shape[1] if block_table.dim() == 2 else block_table.shape[0]
    if int(num_reqs) > 0 and (query_start_loc.numel() < int(num_reqs) + 1 or
                              seq_lens.numel() < int(num_reqs) or
                              (block_table.dim() == 2 and block_table.shape[0] < int(num_reqs))):
        raise ValueError("metadata shorter than num_reqs")
    _check(load().pkv_attention_int8(q.data_ptr(), _rows3(q, "q"), rows, hq, key_cache.data_ptr(),
                                     value_cache.data_ptr(), float(k_scale), float(v_scale), nb,
                                     bs, hkv, d, query_start_loc.data_ptr(), seq_lens.data_ptr(),
                                     block_table.data_ptr(), bt_width, int(num_reqs),
                                     float(scale), out.data_ptr(), _rows3(out, "out"),
                                     _stream(stream)))


def pkv_attention_scored(q, key_cache, value_cache, query_start_loc, seq_lens, block_table,
                         num_reqs, scale, out, softcap=0.0, window=0, alibi_slopes=None,
                         prefix_lens=None, stream=None):
    """pkv_attention with modified scores: softcap * tanh(s / softcap), the
    bias -alibi_slopes[head] * distance (fp32 [Hq]), a sliding window of keys
    and a prefix (int32 [num_reqs]) that every row sees; see include/pkv.h."""
    torch = _torch or _T()
    bf16, i32 = torch.bfloat16, torch.int32
    try:  # (see _write_rope)
        dev = _get_device()
        good = (q.dtype is bf16 and key_cache.dtype is bf16 and value_cache.dtype is bf16 and
                out.dtype is bf16 and query_start_loc.dtype is i32 and seq_lens.dtype is i32 and
                block_table.dtype is i32 and
                dev == q.get_device() == key_cache.get_device() == value_cache.get_device() ==
                out.get_device() == query_start_loc.get_device() == seq_lens.get_device() ==
                block_table.get_device())
        slopes = prefix = 0
        if alibi_slopes is not None:
            good = good and alibi_slopes.dtype is torch.float32 and dev == alibi_slopes.get_device()
            slopes = alibi_slopes.data_ptr()
        if prefix_lens is not None:
            good = good and prefix_lens.dtype is i32 and dev == prefix_lens.get_device()
            prefix = prefix_lens.data_ptr()
    except AttributeError:
        good = False
    if not good:
        _name_culprit((q, "q", bf16), (key_cache, "key_cache", bf16),
                      (value_cache, "value_cache", bf16), (out, "out", bf16),
                      (query_start_loc, "query_start_loc", i32), (seq_lens, "seq_lens", i32),
                      (block_table, "block_table", i32),
                      (alibi_slopes, "alibi_slopes", torch.float32),
                      (prefix_lens, "prefix_lens", i32))
        raise ValueError("arguments must be tensors on the current CUDA device")
    cs = key_cache.shape
    if len(cs) != 4 or cs != value_cache.shape or not (key_cache.is_contiguous() and
                                                       value_cache.is_contiguous()):
        _caches(key_cache, value_cache, bf16)
    nb, bs, hkv, d = cs
    try:
        rows, hq, qd = q.shape
        orows, ohq, od = out.shape
        qs, q1, q2 = q.stride()
        os_, o1, o2 = out.stride()
    except ValueError:
        raise ValueError("q and out must be [rows, num_heads, head_size]") from None
    if orows < rows or ohq != hq or od != d or qd != d:
        raise ValueError("q and out must be [rows, num_heads, %d] with as many rows of out" % d)
    if not (q2 == o2 == 1 and (q1 == o1 == d or hq == 1)):
        raise ValueError("q and out must have contiguous rows")
    if rows == 1:
        qs = os_ = hq * d
    num_reqs, window = int(num_reqs), int(window)
    bts = block_table.shape
    if len(bts) != 2 and (len(bts) != 1 or num_reqs > 1):
        raise ValueError("block_table must be [num_reqs, width]")
    if not (query_start_loc.is_contiguous() and seq_lens.is_contiguous() and
            block_table.is_contiguous()):
        raise ValueError("query_start_loc, seq_lens and block_table must be contiguous")
    if num_reqs > 0 and (query_start_loc.numel() < num_reqs + 1 or seq_lens.numel() < num_reqs or
                         (len(bts) == 2 and bts[0] < num_reqs)):
        raise ValueError("metadata shorter than num_reqs")
    if alibi_slopes is not None and (alibi_slopes.shape != (hq,) or
                                     not alibi_slopes.is_contiguous()):
        raise ValueError("alibi_slopes must be a contiguous [num_heads]")
    if prefix_lens is not None and (prefix_lens.numel() < num_reqs or
                                    not prefix_lens.is_contiguous()):
        raise ValueError("prefix_lens must be contiguous, one per request")
    try:
        args = _SCORED_ARGS.pack(
            q.data_ptr(), qs, rows, key_cache.data_ptr(), value_cache.data_ptr(), nb,
            query_start_loc.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), bts[-1],
            slopes, prefix, out.data_ptr(), os_,
            _raw_stream() if stream is None else _stream(stream), hq, hkv, d, bs, num_reqs,
            window, scale, softcap)
    except (struct.error, OverflowError) as e:
        raise ValueError("an argument is out of range: %s" % e) from None
    rc = (_lib or load()).pkv_attention_scored_packed(args)
    if rc:
        _check(rc)


# The checks of the calls below are one pass of plain attribute reads each, as a small
# call's time is theirs (a list of triples and a helper for each tensor: a call over
# selected pages 13.2 us of host time for 11.9); a failing one is named afterwards.

def _refuse(*named):
    """Raises for the first of these (tensor, name, dtype) that is no tensor of its
    dtype on the current CUDA device."""
    for t, name, _ in named:
        if t is None:
            raise TypeError("%s must be a torch.Tensor" % name)
    _name_culprit(*named)
    raise ValueError("arguments must be tensors on the current CUDA device")


def _cache4(cache):
    sh = cache.shape
    if len(sh) != 3 or sh[2] != INT4_PAGE_BYTES or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous [num_blocks, num_kv_heads, %d]" %
                         INT4_PAGE_BYTES)
    return sh[0], sh[1]


def _head_rows(t, name, heads, d=128):
    """Rows and row stride of a [rows, heads, d] tensor with contiguous rows."""
    try:
        rows, h, w = t.shape
    except ValueError:
        h = w = -1
    if w != d or h != heads:
        raise ValueError("%s must be [rows, %d, %d]" % (name, heads, d))
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and heads != 1):
        raise ValueError("%s must have contiguous rows" % name)
    return rows, heads * d if rows == 1 else s0


def _rows4(k, v, cache, slots, n_tokens, names):
    torch = _torch or _T()
    bf16 = torch.bfloat16
    try:
        good = (k.dtype is bf16 and v.dtype is bf16 and cache.dtype is torch.uint8 and
                slots.dtype is torch.int64 and _get_device() == k.get_device() == v.get_device() ==
                cache.get_device() == slots.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse((k, names[0], bf16), (v, names[1], bf16), (cache, "cache", torch.uint8),
                (slots, names[2], torch.int64))
    nb, hkv = _cache4(cache)
    krows, ks = _head_rows(k, names[0], hkv)
    vrows, vs = _head_rows(v, names[1], hkv)
    if not slots.is_contiguous() or slots.dim() != 1:
        raise ValueError("%s must be contiguous, one-dimensional" % names[2])
    most = slots.shape[0]
    n = most if n_tokens is None else int(n_tokens)
    if n > most or n > krows or n > vrows:
        raise ValueError("n_tokens exceeds the rows of %s/%s/%s" % names)
    return nb, hkv, ks, vs, n


def pkv_write_int4(k, v, cache, slot_mapping, n_tokens=None, stream=None):
    """Quantises k/v ([n, Hkv, 128] bf16) to 4 bits, each row with a scale and a
    zero of its own, into cache ([num_blocks, Hkv, INT4_PAGE_BYTES] uint8) at
    slot_mapping; see include/pkv.h."""
    nb, hkv, ks, vs, n = _rows4(k, v, cache, slot_mapping, n_tokens, ("k", "v", "slot_mapping"))
    rc = (_lib or load()).pkv_write_int4(k.data_ptr(), ks, v.data_ptr(), vs, cache.data_ptr(), nb,
                                         16, hkv, 128, slot_mapping.data_ptr(), n, _stream(stream))
    if rc:
        _check(rc)


def pkv_read_int4(cache, slots, k_out, v_out, n_tokens=None, stream=None):
    """The cached keys and values at slots (int64 [n]; negative: row left as it
    is) as bf16 rows of k_out and v_out ([n, Hkv, 128])."""
    nb, hkv, ks, vs, n = _rows4(k_out, v_out, cache, slots, n_tokens, ("k_out", "v_out", "slots"))
    rc = (_lib or load()).pkv_read_int4(cache.data_ptr(), nb, 16, hkv, 128, slots.data_ptr(), n,
                                        k_out.data_ptr(), ks, v_out.data_ptr(), vs,
                                        _stream(stream))
    if rc:
        _check(rc)


def _step_metadata(query_start_loc, seq_lens, block_table, num_reqs):
    """Checks the step's metadata; returns the width of a block-table row."""
    bts = block_table.shape
    if len(bts) != 2 and (len(bts) != 1 or num_reqs > 1):
        raise ValueError("block_table must be [num_reqs, width]")
    if not (query_start_loc.is_contiguous() and seq_lens.is_contiguous() and
            block_table.is_contiguous()):
        raise ValueError("query_start_loc, seq_lens and block_table must be contiguous")
    if num_reqs > 0 and (query_start_loc.numel() < num_reqs + 1 or seq_lens.numel() < num_reqs or
                         (len(bts) == 2 and bts[0] < num_reqs)):
        raise ValueError("metadata shorter than num_reqs")
    return bts[-1]


def _query_and_out(q, out):
    sh = q.shape
    if len(sh) != 3:
        raise ValueError("q must be [rows, num_heads, head_size]")
    hq = sh[1]
    rows, qs = _head_rows(q, "q", hq)
    orows, os_ = _head_rows(out, "out", hq)
    if orows < rows:
        raise ValueError("out must have as many rows as q")
    if rows == 1:
        os_ = hq * 128
    return rows, hq, qs, os_


def pkv_attention_int4(q, cache, query_start_loc, seq_lens, block_table, num_reqs, scale, out,
                       stream=None):
    """pkv_attention over a cache of 4-bit codes (pkv_write_int4), decodes and
    prompts; see include/pkv.h."""
    torch = _torch or _T()
    bf16, i32 = torch.bfloat16, torch.int32
    try:
        good = (q.dtype is bf16 and cache.dtype is torch.uint8 and out.dtype is bf16 and
                query_start_loc.dtype is i32 and seq_lens.dtype is i32 and
                block_table.dtype is i32 and _get_device() == q.get_device() ==
                cache.get_device() == out.get_device() == query_start_loc.get_device() ==
                seq_lens.get_device() == block_table.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse((q, "q", bf16), (cache, "cache", torch.uint8), (out, "out", bf16),
                (query_start_loc, "query_start_loc", i32), (seq_lens, "seq_lens", i32),
                (block_table, "block_table", i32))
    nb, hkv = _cache4(cache)
    rows, hq, qs, os_ = _query_and_out(q, out)
    num_reqs = int(num_reqs)
    width = _step_metadata(query_start_loc, seq_lens, block_table, num_reqs)
    rc = (_lib or load()).pkv_attention_int4(
        q.data_ptr(), qs, rows, hq, cache.data_ptr(), nb, 16, hkv, 128, query_start_loc.data_ptr(),
        seq_lens.data_ptr(), block_table.data_ptr(), width, num_reqs, float(scale), out.data_ptr(),
        os_, _stream(stream))
    if rc:
        _check(rc)


def _bounds(bounds, nb, hkv, d):
    if bounds.shape != (nb, hkv, 2, d) or not bounds.is_contiguous():
        raise ValueError("bounds must be a contiguous [num_blocks, num_kv_heads, 2, head_size]")


def pkv_page_bounds(key_cache, bounds, slot_mapping, n_tokens=None, stream=None):
    """The smallest and largest keys (bounds: [num_blocks, Hkv, 2, 128] bf16) of
    the pages that the step's tokens (slot_mapping, as in pkv_write) lie in."""
    torch = _torch or _T()
    bf16 = torch.bfloat16
    try:
        good = (key_cache.dtype is bf16 and bounds.dtype is bf16 and
                slot_mapping.dtype is torch.int64 and _get_device() == key_cache.get_device() ==
                bounds.get_device() == slot_mapping.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse((key_cache, "key_cache", bf16), (bounds, "bounds", bf16),
                (slot_mapping, "slot_mapping", torch.int64))
    cs = key_cache.shape
    if len(cs) != 4 or not key_cache.is_contiguous():
        raise ValueError("key_cache must be a contiguous [num_blocks, block_size, Hkv, head_size]")
    nb, bs, hkv, d = cs
    _bounds(bounds, nb, hkv, d)
    if slot_mapping.dim() != 1 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous, one-dimensional")
    n = slot_mapping.shape[0] if n_tokens is None else int(n_tokens)
    if n > slot_mapping.shape[0]:
        raise ValueError("n_tokens exceeds the rows of slot_mapping")
    rc = (_lib or load()).pkv_page_bounds(key_cache.data_ptr(), nb, bs, hkv, d, bounds.data_ptr(),
                                          slot_mapping.data_ptr(), n, _stream(stream))
    if rc:
        _check(rc)


def _lists(sel_table, sel_lens, rows, hkv):
    ss = sel_table.shape
    if len(ss) != 3 or ss[0] < rows or ss[1] != hkv or not sel_table.is_contiguous():
        raise ValueError("sel_table must be a contiguous [rows, num_kv_heads, pages]")
    if sel_lens.dim() != 1 or sel_lens.shape[0] < rows or not sel_lens.is_contiguous():
        raise ValueError("sel_lens must be contiguous, one per row")
    return ss[2]


def pkv_select_pages(q, bounds, query_start_loc, seq_lens, block_table, num_reqs, sel_table,
                     sel_lens, first_pages=0, last_pages=1, stream=None):
    """For each query row and KV head the pages with the best bound on their
    keys' products: their block ids into sel_table ([rows, Hkv, budget] int32),
    the keys in them into sel_lens ([rows] int32); see include/pkv.h."""
    torch = _torch or _T()
    bf16, i32 = torch.bfloat16, torch.int32
    try:
        good = (q.dtype is bf16 and bounds.dtype is bf16 and query_start_loc.dtype is i32 and
                seq_lens.dtype is i32 and block_table.dtype is i32 and sel_table.dtype is i32 and
                sel_lens.dtype is i32 and _get_device() == q.get_device() ==
                bounds.get_device() == query_start_loc.get_device() == seq_lens.get_device() ==
                block_table.get_device() == sel_table.get_device() == sel_lens.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse((q, "q", bf16), (bounds, "bounds", bf16),
                (query_start_loc, "query_start_loc", i32), (seq_lens, "seq_lens", i32),
                (block_table, "block_table", i32), (sel_table, "sel_table", i32),
                (sel_lens, "sel_lens", i32))
    sh = bounds.shape
    if len(sh) != 4 or sh[2] != 2 or not bounds.is_contiguous():
        raise ValueError("bounds must be a contiguous [num_blocks, num_kv_heads, 2, head_size]")
    nb, hkv, _, d = sh
    sh = q.shape
    if len(sh) != 3:
        raise ValueError("q must be [rows, num_heads, head_size]")
    hq = sh[1]
    rows, qs = _head_rows(q, "q", hq)
    budget = _lists(sel_table, sel_lens, rows, hkv)
    num_reqs = int(num_reqs)
    width = _step_metadata(query_start_loc, seq_lens, block_table, num_reqs)
    rc = (_lib or load()).pkv_select_pages(
        q.data_ptr(), qs, rows, hq, bounds.data_ptr(), nb, 16, hkv, d,
        query_start_loc.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), width, num_reqs,
        budget, int(first_pages), int(last_pages), sel_table.data_ptr(), sel_lens.data_ptr(),
        _stream(stream))
    if rc:
        _check(rc)


def pkv_reserve_select(max_q_rows, block_table_width, num_kv_heads):
    """Sizes the workspace of pkv_select_pages, as pkv_reserve_workspace does the
    other one (needed before a CUDA-graph capture)."""
    _check(load().pkv_reserve_select(int(max_q_rows), int(block_table_width), int(num_kv_heads)))


def pkv_attention_selected(q, key_cache, value_cache, sel_table, sel_lens, scale, out,
                           stream=None):
    """Attention of each query row over the pages listed for it and each KV head
    (pkv_select_pages); see include/pkv.h."""
    torch = _torch or _T()
    bf16, i32 = torch.bfloat16, torch.int32
    try:
        good = (q.dtype is bf16 and key_cache.dtype is bf16 and value_cache.dtype is bf16 and
                sel_table.dtype is i32 and sel_lens.dtype is i32 and out.dtype is bf16 and
                _get_device() == q.get_device() == key_cache.get_device() ==
                value_cache.get_device() == sel_table.get_device() == sel_lens.get_device() ==
                out.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse((q, "q", bf16), (key_cache, "key_cache", bf16),
                (value_cache, "value_cache", bf16), (sel_table, "sel_table", i32),
                (sel_lens, "sel_lens", i32), (out, "out", bf16))
    sh = key_cache.shape
    if len(sh) != 4 or not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, head_size]")
    if sh != value_cache.shape:
        raise ValueError("key_cache and value_cache shapes differ")
    nb, bs, hkv, d = sh
    rows, hq, qs, os_ = _query_and_out(q, out)
    width = _lists(sel_table, sel_lens, rows, hkv)
    rc = (_lib or load()).pkv_attention_selected(
        q.data_ptr(), qs, rows, hq, key_cache.data_ptr(), value_cache.data_ptr(), nb, bs, hkv, d,
        sel_table.data_ptr(), width, sel_lens.data_ptr(), float(scale), out.data_ptr(), os_,
        _stream(stream))
    if rc:
        _check(rc)


def pkv_plan(q_rows, num_heads, num_kv_heads, query_start_loc, seq_lens, block_table_width,
             num_reqs, stream=None):
    """Builds one step plan on the current device, for pkv_attention_planned
    calls (one per layer) that follow it; see include/pkv.h."""
    import torch
    for t, n in ((query_start_loc, "query_start_loc"), (seq_lens, "seq_lens")):
        _require(t, torch.int32, n)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    if int(num_reqs) > 0 and (query_start_loc.numel() < int(num_reqs) + 1 or
                              seq_lens.numel() < int(num_reqs)):
        raise ValueError("metadata shorter than num_reqs")
    _check(load().pkv_plan(int(q_rows), int(num_heads), int(num_kv_heads),
                           query_start_loc.data_ptr(), seq_lens.data_ptr(),
                           int(block_table_width), int(num_reqs), _stream(stream)))


def pkv_attention_planned(q, key_cache, value_cache, block_table, scale, out, stream=None):
    """One layer's attention on the current step plan (pkv_plan)."""
    torch = _T()
    if not (_all_on_device(torch.bfloat16, q, key_cache, value_cache, out) and
            _all_on_device(torch.int32, block_table)):
        for t, n in ((q, "q"), (key_cache, "key_cache"), (value_cache, "value_cache"),
                     (out, "out")):
            _require(t, torch.bfloat16, n)
        _require(block_table, torch.int32, "block_table")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    nb, bs, hkv, d = _caches(key_cache, value_cache, torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [rows, num_heads, head_size]")
    rows, hq, _ = q.shape
    if out.shape[0] < rows or _per_row(out) != hq * d:
        raise ValueError("out must hold [rows, num_heads * head_size]")
    _check(load().pkv_attention_planned(q.data_ptr(), _rows3(q, "q"), hq, key_cache.data_ptr(),
                                        value_cache.data_ptr(), nb, bs, hkv, d,
                                        block_table.data_ptr(), float(scale), out.data_ptr(),
                                        _rows3(out, "out"), _stream(stream)))


def pkv_reserve_workspace(max_reqs, max_q_rows, block_table_width, num_heads, num_kv_heads):
    _check(load().pkv_reserve_workspace(int(max_reqs), int(max_q_rows), int(block_table_width),
                                        int(num_heads), int(num_kv_heads)))


class WorkspaceInfo(ctypes.Structure):
    """Mirror of pkv_workspace_info (include/pkv.h)."""
    _fields_ = [("bytes", ctypes.c_int64), ("decode_units", ctypes.c_int64),
                ("prefill_tiles", ctypes.c_int64), ("split_pairs", ctypes.c_int64),
                ("partial_rows", ctypes.c_int64), ("decode_workers", ctypes.c_int32),
                ("decode_workers_int8", ctypes.c_int32)]


def pkv_workspace_size(max_reqs, max_q_rows, block_table_width, num_heads, num_kv_heads,
                       num_sms) -> dict:
    """Bytes and plan capacities of the workspace pkv_reserve_workspace would
    hold for these sizes on a device with num_sms SMs (host-only)."""
    L = load()
    fn = L.pkv_workspace_size
    if fn.argtypes is None:
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                       ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(WorkspaceInfo)]
    info = WorkspaceInfo()
    _check(fn(int(max_reqs), int(max_q_rows), int(block_table_width), int(num_heads),
              int(num_kv_heads), int(num_sms), ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in WorkspaceInfo._fields_}


def pkv_get_error(stream=None) -> int:
    """Synchronises the stream; returns and clears the device error words
    (the allocating calls' and pkv_attention_noalloc's)."""
    bits = ctypes.c_int32(0)
    _check(load().pkv_get_error(_stream(stream), ctypes.byref(bits)))
    return bits.value


def pkv_num_sms() -> int:
    return load().pkv_num_sms()


def pkv_trace_enable(on: bool) -> None:
    load().pkv_trace_enable(1 if on else 0)


def pkv_trace_read():
    """{kind: (total ms, launches)} of the traced launches since the last read."""
    n = len(TRACE_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    rc = load().pkv_trace_read(ms, cnt, n)
    if rc < 0:
        _check(rc)
    return {k: (ms[i], cnt[i]) for i, k in enumerate(TRACE_KINDS)}


def pkv_launch_count() -> int:
    return load().pkv_launch_count()


def pkv_attention_noalloc(q, key_cache, value_cache, query_start_loc, seq_lens, block_table,
                          num_reqs, scale, out, stream=None):
    """pkv_attention computed with the library's static scratch array instead
    of a cudaMalloc'd workspace, for callers that cannot allocate device
    memory (see include/pkv.h).  Same arguments and result; raises PkvError
    with the return code when a host check refuses the call."""
    import torch
    L = load()
    fn = L.pkv_attention_noalloc
    if fn.argtypes is None:
        i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, i64, i64, i32, vp, vp, i64, i32, i32, i32, vp, vp, vp, i64, i32, f32,
                       vp, i64, vp]
    for t, n in ((q, "q"), (key_cache, "key_cache"), (value_cache, "value_cache"), (out, "out")):
        _require(t, torch.bfloat16, n)
    for t, n in ((query_start_loc, "query_start_loc"), (seq_lens, "seq_lens"),
                 (block_table, "block_table")):
        _require(t, torch.int32, n)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()) or key_cache.dim() != 4:
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, head_size]")
    nb, bs, hkv, d = key_cache.shape
    rows, hq, _ = q.shape
    bt_width = block_table.shape[1] if block_table.dim() == 2 else block_table.shape[0]
    rc = fn(q.data_ptr(), _rows3(q, "q"), rows, hq, key_cache.data_ptr(), value_cache.data_ptr(),
            nb, bs, hkv, d, query_start_loc.data_ptr(), seq_lens.data_ptr(),
            block_table.data_ptr(), bt_width, int(num_reqs), float(scale), out.data_ptr(),
            _rows3(out, "out"), _stream(stream))
    if rc != 0:
        raise PkvError(rc, "pkv_attention_noalloc refused the call")


def pkv_prepare_step(query_start_loc, num_computed, persistent_block_table, num_reqs,
                     num_tokens_padded, positions, seq_lens, slot_mapping, block_table=None,
                     idx_mapping=None, stream=None):
    """Positions, seq_lens, slot mapping and the batch-order block table on
    the device (see include/pkv.h)."""
    import torch
    L = load()
    fn = L.pkv_prepare_step
    if fn.argtypes is None:
        i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, vp, vp, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp]
    for t, n, dt in ((query_start_loc, "query_start_loc", torch.int32),
                     (num_computed, "num_computed", torch.int32),
                     (persistent_block_table, "persistent_block_table", torch.int32),
                     (positions, "positions", torch.int64), (seq_lens, "seq_lens", torch.int32),
                     (slot_mapping, "slot_mapping", torch.int64)):
        _require(t, dt, n)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % n)
    if block_table is not None:
        _require(block_table, torch.int32, "block_table")
    if idx_mapping is not None:
        _require(idx_mapping, torch.int32, "idx_mapping")
    rows, width = persistent_block_table.shape
    _check(fn(query_start_loc.data_ptr(), num_computed.data_ptr(),
              idx_mapping.data_ptr() if idx_mapping is not None else None,
              persistent_block_table.data_ptr(), rows, width, int(num_reqs),
              int(num_tokens_padded), positions.data_ptr(), seq_lens.data_ptr(),
              slot_mapping.data_ptr(), block_table.data_ptr() if block_table is not None else None,
              _stream(stream)))
