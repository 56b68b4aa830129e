"""The argument checks of the calls around the attention, without a GPU:
ac_layer.cu linked with stand-ins for the CUDA runtime and the kernels
(layer_stub.cu, cudart_stub.c).  Every refusal launches nothing; what passes reaches the
launcher with the sizes that the arguments say."""
import ctypes
import math
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "clustered_sparse_attention_head_b200", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from clustered_sparse_attention_head_b200 import _abi, _build
    out = str(tmp_path_factory.mktemp("stub") / "libstub.so")
    subprocess.check_call([_build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1", "-Xcompiler",
                           "-fPIC", "-Xlinker", "-Bsymbolic", "-shared", "-cudart", "none",
                           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "ac_layer.cu"),
                           os.path.join(ROOT, "tests", "layer_stub.cu"),
                           os.path.join(ROOT, "tests", "cudart_stub.c"), "-o", out])
    L = ctypes.CDLL(out)
    for name, (args, res) in _abi.SIGNATURES.items():
        if name.startswith(("ac_layer", "ac_rope", "ac_qk", "ac_cache")):
            getattr(L, name).argtypes, getattr(L, name).restype = args, res
    L.stub_freq.restype = ctypes.c_double
    return L


def _cfg(**over):
    from clustered_sparse_attention_head_b200.layer import LayerConfig
    base = dict(heads=4, kv_heads=2, d=64, norm="rms", rope_dims=(16, 24), rope_max=(5, 7), page_size=16, causal_block=1)
    base.update(over)
    return LayerConfig(**base).to_c()


def _create(lib, **over):
    h = ctypes.c_void_p()
    raw = {k: over.pop(k) for k in list(over) if k.startswith("c_")}
    c = _cfg(**over)
    for k, v in raw.items():
        setattr(c, k[2:], v)
    code = lib.ac_layer_create(ctypes.byref(c), ctypes.byref(h))
    return code, h


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


@pytest.mark.parametrize("over, code", [
    (dict(), OK),
    (dict(heads=5), INVALID), (dict(c_heads=0), INVALID), (dict(c_kv_heads=0), INVALID), (dict(heads=8192, kv_heads=1), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(c_dtype=5), INVALID), (dict(c_w_dtype=-1), INVALID), (dict(c_norm=9), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=0.0), OK),
    (dict(c_rope_axes=4), INVALID), (dict(c_rope_axes=-1), INVALID), (dict(rope_dims=(), rope_max=()), OK),
    (dict(rope_dims=(15, 24)), INVALID), (dict(rope_dims=(0, 24)), INVALID), (dict(rope_dims=(48, 24)), INVALID),
    (dict(rope_max=(0, 7)), INVALID), (dict(rope_theta=0.0), INVALID), (dict(rope_theta=math.inf), INVALID),
    (dict(c_rope_layout=3), INVALID), (dict(c_rope_scaling=7), INVALID),
    (dict(rope_layout="half", rope_dims=(16, 24)), UNSUPPORTED), (dict(rope_layout="half", rope_dims=(16, 16)), OK),
    (dict(rope_scaling="linear", rope_factor=0.5), INVALID), (dict(rope_scaling="ntk", rope_dims=(2, 24), rope_factor=2.0), INVALID),
    (dict(rope_scaling="yarn", rope_factor=2.0, rope_orig=0), INVALID),
    (dict(rope_scaling="yarn", rope_factor=2.0, rope_orig=64, rope_beta_fast=1.0), INVALID),
    (dict(rope_scaling="yarn", rope_factor=2.0, rope_orig=64), OK),
    (dict(rope_dims=(64,), rope_max=(1 << 27,)), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED), (dict(page_size=-16), INVALID),
    (dict(causal_block=-1), INVALID), (dict(window=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
])
def test_layer_config(lib, over, code):
    got, h = _create(lib, **over)
    assert got == code
    assert bool(h.value) == (code == OK)
    if h.value:
        lib.ac_layer_destroy(h)


def test_config_python_refusals():
    for over in (dict(norm="batch"), dict(dtype="f16"), dict(rope_layout="spiral"), dict(rope_scaling="x"),
                 dict(rope_dims=(16,)), dict(rope_dims=(2, 2, 2, 2), rope_max=(1, 1, 1, 1))):
        with pytest.raises(ValueError):
            _cfg(**over)


def _buf():
    raw = ctypes.create_string_buffer(1 << 16)
    return raw, (ctypes.addressof(raw) + 255) // 256 * 256


def _view(data, sb, sn, sh):
    from clustered_sparse_attention_head_b200 import _abi
    return _abi.ac_tensor(data, sb, sn, sh)


def test_norm_rope_checks(lib):
    code, h = _create(lib)
    raw, base = _buf()
    keep = [raw]
    n = 6

    def call(q="ok", qo="ok", batch=2, n=n, table=base, pos=None, pos_stride=0, k=None, ko=None):
        q = _view(base, n * 256, 256, 64) if q == "ok" else q
        qo = _view(base + 16384, n * 256, 64, n * 64) if qo == "ok" else qo
        keep.extend([q, qo])
        ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
        before = lib.stub_launches()
        code = lib.ac_qk_norm_rope(h, batch, n, table, pos, pos_stride, ref(q), None, None, ref(qo), ref(k), None, None,
                                   ref(ko), None)
        return code, lib.stub_launches() - before

    assert call() == (OK, 1)
    assert [lib.stub_rows(i) for i in range(3)] == [1, 2, n]
    assert lib.stub_rows(5) == 20 and lib.stub_rows(6) == 35 and lib.stub_rows(7) == 5 * 8
    assert call(k=_view(base, 6 * 256, 256, 64), ko=_view(base + 32768, 6 * 128, 64, 6 * 64)) == (OK, 1)
    assert lib.stub_rows(0) == 2
    assert call(batch=0) == (OK, 0) and call(n=0) == (OK, 0)
    assert call(qo=_view(base, 6 * 256, 256, 64)) == (OK, 1)                      # in place
    assert call(q=_view(base, 0, 0, 64)) == (OK, 1)                               # a broadcast input
    for bad in (dict(batch=-1), dict(n=-1), dict(table=None), dict(table=base + 4), dict(qo=None), dict(q=None),
                dict(q=_view(None, 1536, 256, 64)), dict(q=_view(base + 2, 1536, 256, 64)),
                dict(q=_view(base, 1536, 256, 68)), dict(q=_view(base, -1536, 256, 64)),
                dict(q=_view(base, 1 << 41, 256, 64)), dict(q=_view(base, 0, 1 << 31, 64)),
                dict(q=_view(base, 0, 256, 1 << 31)),
                dict(qo=_view(base + 16384, 0, 64, 384)), dict(qo=_view(base + 16384, 1536, 0, 64)),
                dict(qo=_view(base + 16384, 1536, 32, 384)), dict(qo=_view(base + 16384, 1536, 64, 128)),
                dict(qo=_view(base + 512, 1536, 256, 64)),                        # one token further: overlaps
                dict(qo=_view(base, 1536, 64, 384)),                              # the input's memory, other strides
                dict(pos=base, pos_stride=-3), dict(k=_view(base, 1536, 256, 64))):
        assert call(**bad) == (INVALID, 0), bad
    assert call(batch=1 << 16, n=1 << 16, q=_view(base, 0, 0, 64))[0] == UNSUPPORTED
    # strides of dimensions of one element are not read
    code1, h1 = _create(lib, heads=1, kv_heads=1)
    t = _view(base, -7, 3, 5)
    u = _view(base + 4096, -7, 3, 5)
    assert lib.ac_qk_norm_rope(h1, 1, 1, base, None, 0, ctypes.byref(t), None, None, ctypes.byref(u), None, None, None,
                               None, None) == OK
    lib.stub_device(3)  # another current device than the layer's
    assert call() == (INVALID, 0)
    lib.stub_device(0)
    assert call() == (OK, 1)


def test_backward_checks(lib):
    code, h = _create(lib)
    need = ctypes.c_size_t()
    lib.ac_layer_workspace_size(h, ctypes.byref(need))
    raw, base = _buf()
    keep = [raw]

    def call(h=h, g="ok", x="ok", dx="ok", dw=base + 60000 // 256 * 256, db=None, ws=base + 32768, have=None, n=6):
        g = _view(base, 1536, 64, 384) if g == "ok" else g
        x = _view(base + 8192, 1536, 256, 64) if x == "ok" else x
        dx = _view(base + 16384, 1536, 256, 64) if dx == "ok" else dx
        keep.extend([g, x, dx])
        ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
        before = lib.stub_launches()
        code = lib.ac_qk_norm_rope_backward(h, 2, n, base, None, 0, ref(g), ref(x), None, ref(dx), dw, db, None, None,
                                            None, None, None, None, ws, need.value if have is None else have, None)
        return code, lib.stub_launches() - before

    assert call() == (OK, 1)
    assert call(dx=_view(base, 1536, 64, 384)) == (OK, 1)          # over the upstream gradient
    assert call(dw=None, ws=None, have=0) == (OK, 1)               # no sums, no workspace
    assert call(ws=None) == (WORKSPACE, 0) and call(have=need.value - 1) == (WORKSPACE, 0)
    assert call(ws=base + 8) == (WORKSPACE, 0)
    for bad in (dict(g=None), dict(dx=None), dict(x=None), dict(g=None, dx=None),
                dict(dx=_view(base + 16384, 1536, 0, 64)), dict(dx=_view(base + 8192 + 128, 1536, 256, 64))):
        assert call(**bad)[0] == INVALID, bad
    # no tokens: the sums are zero
    ctypes.memset(base + 59904, 1, 128)
    assert call(n=0, dw=base + 59904) == (OK, 0)
    assert ctypes.string_at(base + 59904, 128) == bytes(128)
    _, plain = _create(lib, norm="none")
    assert call(h=plain, x=None, dw=None, ws=None, have=0) == (OK, 1)
    assert call(h=plain) == (INVALID, 0)                           # no weight, no gradient of it


def test_cache_checks(lib):
    code, h = _create(lib)
    need = ctypes.c_size_t()
    lib.ac_layer_workspace_size(h, ctypes.byref(need))
    raw, base = _buf()
    keep = [raw]
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731

    def attn(h=h, seqs=2, tokens=5, max_q=5, max_kv=40, q_start=base, kv_len=base, table=base, max_pages=3, num_pages=4,
             q="ok", k=base, v=base, out="ok", ws=base, have=None):
        q = _view(base, 0, 256, 64) if q == "ok" else q
        out = _view(base + 8192, 0, 256, 64) if out == "ok" else out
        keep.extend([q, out])
        before = lib.stub_launches()
        code = lib.ac_cache_attn(h, seqs, tokens, max_q, max_kv, q_start, kv_len, table, max_pages, num_pages, ref(q), k, v,
                                 ref(out), None, ws, need.value if have is None else have, None)
        return code, lib.stub_launches() - before

    assert attn() == (OK, 1)
    assert [lib.stub_attn(i) for i in range(6)] == [5, 40, 2, 4, 1, 0]
    assert attn(max_kv=1000, max_q=99) == (OK, 1) and lib.stub_attn(1) == 48 and lib.stub_attn(0) == 5
    assert attn(num_pages=0, k=None, v=None) == (OK, 1) and lib.stub_attn(1) == 0
    assert attn(seqs=0) == (OK, 0) and attn(tokens=0) == (OK, 0) and attn(max_q=0) == (OK, 0)
    for bad in (dict(seqs=-1), dict(tokens=-1), dict(max_q=-1), dict(max_kv=-1), dict(max_pages=-1), dict(num_pages=-1),
                dict(q_start=None), dict(kv_len=None), dict(table=None), dict(k=None), dict(v=base + 8), dict(q=None),
                dict(out=None), dict(out=_view(base + 8192, 0, 0, 64)), dict(out=_view(base + 8200, 0, 256, 64)),
                dict(out=_view(base + 512, 0, 256, 64))):
        assert attn(**bad) == (INVALID, 0), bad
    assert attn(ws=None) == (WORKSPACE, 0) and attn(have=need.value - 1) == (WORKSPACE, 0)
    assert attn(q=_view(base, 0, 0, 64)) == (UNSUPPORTED, 0)              # a broadcast query
    assert attn(num_pages=1 << 26) == (UNSUPPORTED, 0)                    # 2^31 rows of a pool
    assert attn(num_pages=(1 << 26) - 1) == (OK, 1)
    _, none = _create(lib, page_size=0)
    assert attn(h=none) == (UNSUPPORTED, 0)
    _, f32 = _create(lib, dtype="f32")
    assert attn(h=f32) == (UNSUPPORTED, 0)
    _, wide = _create(lib, heads=129, kv_heads=1)
    assert attn(h=wide, q=_view(base, 0, 129 * 64, 64), out=_view(base + 32768, 0, 129 * 64, 64), tokens=1) == (UNSUPPORTED, 0)

    def append(h=h, seqs=2, tokens=5, q="ok", qo="ok", k="ok", v="ok", table=base, num_pages=4, pages=base):
        q = _view(base, 0, 256, 64) if q == "ok" else q
        qo = _view(base + 8192, 0, 256, 64) if qo == "ok" else qo
        k = _view(base, 0, 128, 64) if k == "ok" else k
        v = _view(base, 0, 128, 64) if v == "ok" else v
        keep.extend([q, qo, k, v])
        before = lib.stub_launches()
        code = lib.ac_cache_append(h, seqs, tokens, base, base, base, 3, num_pages, table, None, ref(k), None, None, ref(v),
                                   pages, pages, ref(q), None, None, ref(qo), None)
        return code, lib.stub_launches() - before

    assert append() == (OK, 1)
    assert [lib.stub_rows(i) for i in (0, 1, 2, 3, 4)] == [3, 1, 5, 2, 4]
    assert append(q=None, qo=None) == (OK, 1) and lib.stub_rows(0) == 2
    assert append(tokens=0) == (OK, 0) and append(seqs=0) == (OK, 0)
    for bad in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(table=None), dict(pages=None),
                dict(pages=base + 2), dict(v=_view(base, 0, 100, 64)), dict(seqs=-2)):
        assert append(**bad) == (INVALID, 0), bad
    assert append(h=none) == (UNSUPPORTED, 0)


def test_table_and_frequencies(lib):
    """Sizes and frequencies of the table: the pairs' axes, and the three scalings."""
    code, h = _create(lib, rope_scaling="yarn", rope_factor=4.0, rope_orig=100, rope_theta=100.0, rope_beta_fast=8.0,
                      rope_beta_slow=1.0)
    nb = ctypes.c_size_t()
    assert lib.ac_rope_table_size(h, ctypes.byref(nb)) == OK and nb.value == 8 * (5 * 8 + 7 * 12)
    raw, base = _buf()
    assert lib.ac_rope_table(h, base, None) == OK
    assert lib.ac_rope_table(h, base + 4, None) == INVALID and lib.ac_rope_table(h, None, None) == INVALID
    assert lib.stub_freq(-1) == pytest.approx(0.1 * math.log(4) + 1, rel=1e-15)
    for pair, (j, dim) in ((0, (0, 16)), (3, (3, 16)), (8, (0, 24)), (19, (11, 24))):
        f = 100.0 ** (-2 * j / dim)
        keep = min(1.0, max(0.0, (100 * f / (2 * math.pi) - 1) / 7))
        assert lib.stub_freq(pair) == pytest.approx(f * keep + f / 4 * (1 - keep), rel=1e-14)
    _, plain = _create(lib, rope_dims=(), rope_max=())
    assert lib.ac_rope_table_size(plain, ctypes.byref(nb)) == UNSUPPORTED
    assert lib.ac_rope_table(plain, base, None) == UNSUPPORTED
