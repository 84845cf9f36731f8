"""Host-side checks of the operators of include/mosaic_ops.h: refusals before any launch,
sizes, and the cache layout's text (each byte of a record used once)."""
import ctypes
import os
import re

import pytest
import torch

import ops_ref as ref
from bit_quantized_gemm_zipperengine_b200 import build


@pytest.fixture(scope="module")
def L():
    from bit_quantized_gemm_zipperengine_b200 import build, mosaic
    build.build()
    return mosaic.lib()


@pytest.fixture(scope="module")
def buf():
    """Real buffers (device memory with a GPU, host memory without, where nothing can launch)."""
    keep, dev = [], "cuda" if torch.cuda.is_available() else "cpu"

    def make(nbytes, offset=0):
        t = torch.zeros(nbytes + 256, dtype=torch.uint8, device=dev)
        keep.append(t)
        return -(-t.data_ptr() // 128) * 128 + offset

    return make


def heads(ptr, n, st, sh):
    a = (ctypes.c_int64 * 4)(ptr, n, st, sh)
    return a


def test_layout_uses_every_byte_once():
    for D in (64, 128):
        used = set()
        for i in range(16):
            for d in range(D):
                kc, vc, ks, vs = ref.record_bytes(i, d, D)
                used |= {kc, vc, ks, vs}
        assert used == set(range(18 * D))


def test_cache_bytes(L):
    assert L.mq_kv_cache_bytes(3, 64, 8, 128) == 3 * 64 * 8 * 144
    assert L.mq_kv_cache_bytes(1 << 20, 128, 8, 128) == (1 << 20) * 128 * 8 * 144  # past 32 bits
    for bad in ((0, 16, 1, 64), (1, 8, 1, 64), (1, 24, 1, 64), (1, 16, 0, 64), (1, 16, 1, 96), (1, 16, 1, 256)):
        assert L.mq_kv_cache_bytes(*bad) == 0
    assert L.mq_kv_attention_workspace_bytes(8, 3, 128, 1) == 0
    assert L.mq_kv_attention_workspace_bytes(8, 2, 96, 1) == 0
    assert L.mq_kv_attention_workspace_bytes(8, 2, 128, 0) == 0


def test_gemv_refusals(L, buf):
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    N, K, M = 128, 256, 4
    w = mosaic.NVFP4Mat(N, K, buf(N * K // 2), None, buf(N * K // 16), buf(4))
    r = mosaic.ResidualPacked(N, K, 2, buf(4096), buf(1024), buf(8), buf(12), buf(8))
    X, Y = buf(17 * K * 2), buf(17 * N * 2)

    n = L.mq_gemv_workspace_bytes(M, K)
    ws = buf(n)
    assert n > 0 and L.mq_gemv_workspace_bytes(17, K) == 0 and L.mq_gemv_workspace_bytes(0, K) == 0
    assert L.mq_gemv_workspace_bytes(1, 96) == 0

    def call(X=X, ty=0, ldx=K, w=w, r=None, Y=Y, ldy=N, M=M, N=N, K=K, flags=0, ws=ws, n=n):
        return L.mq_gemv(X, ty, ldx, ctypes.byref(w) if w else None, ctypes.byref(r) if r else None, Y, ldy, M, N, K, flags, ws, n, None)

    assert call(X=None) == 1 and call(Y=None) == 1 and call(w=None) == 1 and call(ty=2) == 1
    assert call(M=0) == 1 and call(N=96) == 1 and call(K=96) == 1 and call(N=192) == 1
    assert call(ldx=K - 8) == 1 and call(ldx=K + 4) == 1 and call(ldy=N - 1) == 1
    assert call(X=X + 8) == 1 and call(Y=Y + 1) == 1
    assert call(flags=2) == 1 and call(flags=4 | 8) == 1 and call(flags=16) == 1
    assert call(M=17) == 2
    assert call(ws=None) == 3 and call(n=n - 1) == 3 and call(ws=ws + 8) == 3
    assert call(r=mosaic.ResidualPacked(N, K, 2, buf(4096), buf(1024), None, buf(12), None)) == 1
    assert call(r=mosaic.ResidualPacked(N, 2 * K, 2, *[getattr(r, f) for f in ("blk_codes", "blk_sf", "blk_kt", "tile_ptr", "bitmap")])) == 1
    assert call(w=mosaic.NVFP4Mat(N, K, w.codes, None, None, w.gscale)) == 1
    assert call(w=mosaic.NVFP4Mat(N, K, w.codes + 8, None, w.sf_swz, w.gscale)) == 1


def test_gemv_refuses_more_rows_than_a_grid_counts(L, buf):
    """Before any launch: a launch that fails would leave its error for the next CUDA call."""
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    p, K = buf(1 << 12), 64
    for N, want in ((64 * 65536, 2), (2 ** 31 - 64, 2)):
        w = mosaic.NVFP4Mat(N, K, p, None, p, p)
        n = L.mq_gemv_workspace_bytes(1, K)
        assert L.mq_gemv(p, 0, K, ctypes.byref(w), None, p, N, 1, N, K, 0, p, n, None) == want


def test_rope_and_append_refusals(L, buf):
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    T, D = 4, 64
    mem = buf(1 << 16)
    h = heads(mem, 2, 2 * D, D)
    pos, freq, slots = buf(8 * T), buf(8 * D), buf(8 * T)

    def rope(q=h, k=h, qo=h, ko=h, T=T, D=D, ty=0, wq=None, wk=None, eps=1e-6, pos=pos, freq=freq, rot=64):
        return L.mq_qk_norm_rope(q, k, qo, ko, T, D, ty, wq, wk, eps, pos, freq, rot, 0, None)

    assert rope(q=None) == 1 and rope(k=None) == 1 and rope(q=None, k=None, qo=None, ko=None) == 1
    assert rope(T=-1) == 1 and rope(D=96) == 1 and rope(ty=7) == 1
    assert rope(rot=72) == 1 and rope(rot=80) == 1 and rope(rot=-16) == 1 and rope(pos=None) == 1 and rope(freq=None) == 1
    assert rope(eps=-1.0) == 1 and rope(eps=float("nan")) == 1 and rope(wq=mem + 2) == 1
    for bad in (heads(mem + 2, 2, 2 * D, D), heads(mem, 2, 2 * D + 4, D), heads(mem, 2, 2 * D, D + 4), heads(mem, 0, 2 * D, D),
                heads(mem, 2, -2 * D, D), heads(0, 2, 2 * D, D)):
        assert rope(q=bad) == 1 and rope(qo=bad) == 1
    assert rope(qo=heads(mem, 2, 2 * D, 0)) == 1 and rope(qo=heads(mem, 2, 0, D)) == 1  # rows that overlap
    assert rope(qo=heads(mem, 3, 3 * D, D)) == 1                                        # other heads than q's
    assert rope(T=0, q=heads(0, 2, 0, 0), k=None, qo=heads(0, 2, 0, 0), ko=None) == 0   # nothing to do

    pages = buf(4 * 2 * 2 * 1152)
    c = mosaic.KVCacheStruct(pages, 4, 32, 2, 64, None, None)

    def app(k=h, v=h, T=T, ty=0, slots=slots, c=c):
        return L.mq_kv_append(k, v, T, ty, slots, ctypes.byref(c) if c else None, None)

    def read(k=h, v=h, T=T, ty=0, slots=slots, c=c):
        return L.mq_kv_read(ctypes.byref(c) if c else None, slots, T, k, v, ty, None)

    for f in (app, read):
        assert f(k=None) == 1 and f(v=None) == 1 and f(T=-2) == 1 and f(ty=-1) == 1 and f(slots=None) == 1 and f(c=None) == 1
        assert f(k=heads(mem, 3, 3 * D, D)) == 1 and f(v=heads(mem, 1, D, D)) == 1
        for bad in ((pages, 4, 24, 2, 64), (pages, 0, 32, 2, 64), (pages + 64, 4, 32, 2, 64), (None, 4, 32, 2, 64), (pages, 4, 32, 2, 256)):
            assert f(c=mosaic.KVCacheStruct(*bad, None, None)) == 1
        assert f(T=0) == 0
    assert read(k=heads(mem, 2, 2 * D, 0)) == 1

    def both(q=h, k=h, v=h, qo=h, ko=None, slots=slots, c=c, rot=64):
        return L.mq_qkv_append(q, k, v, qo, ko, T, 0, None, None, 1e-6, pos, freq, rot, 0, slots, ctypes.byref(c), None)

    assert both(q=None) == 1 and both(k=None) == 1 and both(v=None) == 1 and both(qo=None) == 1 and both(slots=None) == 1
    assert both(rot=24) == 1 and both(k=heads(mem, 1, D, D)) == 1 and both(ko=heads(mem, 1, D, D)) == 1


def test_outputs_whose_rows_overlap_are_refused(L, buf):
    T, D, mem = 4, 64, buf(1 << 14)
    q = heads(mem, 3, 3 * D, D)

    def rope(qo, T=T, q=q):
        return L.mq_qk_norm_rope(q, None, qo, None, T, D, 0, None, None, 1e-6, None, None, 0, 0, None)

    for token, head in ((D, D), (2 * D, D), (3 * D - 8, D), (D, 4 * D - 8), (D, 3 * D), (3 * D, D - 8), (D - 8, 8 * D)):
        assert rope(heads(mem, 3, token, head)) == 1, (token, head)
    assert rope(heads(mem, 3, 0, D - 8), T=1) == 1 and rope(heads(mem, 1, D - 8, 0), q=heads(mem, 1, D, D)) == 1


def test_attention_refusals(L, buf):
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    T, D, B = 3, 64, 3
    q, o = heads(buf(1 << 14), 4, 4 * D, D), heads(buf(1 << 14), 4, 4 * D, D)
    c = mosaic.KVCacheStruct(buf(4 * 2 * 2 * 1152), 4, 32, 2, 64, None, None)
    table, lens, cu = buf(4 * B * 4), buf(4 * B), buf(16)
    n = L.mq_kv_attention_workspace_bytes(4, 2, 64, 1)
    ws = buf(max(n, 16))

    def call(q=q, o=o, T=T, ty=0, c=c, table=table, stride=4, pages=4, B=B, cu=cu, mq=1, lens=lens, scale=0.1, window=0, ws=ws, n=n):
        return L.mq_kv_attention(q, o, None, T, ty, ctypes.byref(c) if c else None, table, stride, pages, B, cu, mq, lens, scale, window,
                                 ws, n, None)

    assert call(q=None) == 1 and call(o=None) == 1 and call(c=None) == 1 and call(table=None) == 1 and call(lens=None) == 1
    assert call(T=-1) == 1 and call(B=-1) == 1 and call(ty=2) == 1 and call(mq=0) == 1 and call(window=-1) == 1
    assert call(scale=float("inf")) == 1 and call(scale=float("nan")) == 1
    assert call(stride=3) == 1 and call(pages=0) == 1 and call(cu=None, B=2) == 1
    assert call(q=heads(q[0], 3, 3 * D, D), o=heads(o[0], 3, 3 * D, D)) == 1
    assert call(o=q) == 1 and call(o=heads(o[0], 4, 4 * D, 0)) == 1 and call(o=heads(o[0], 2, 4 * D, D)) == 1
    if n:
        assert call(ws=None) == 3 and call(n=n - 1) == 3 and call(ws=ws + 8) == 3
    assert call(T=0) == 0 and call(B=0) == 0


def test_read_only_loads_are_of_final_data_alone():
    """The operators' kernels, and the quantizer of prompts, start before their predecessor ends. __ldg promises that what it reads
    does not change while the kernel lives: only the packed weight, whose writers ended before."""
    csrc = os.path.join(build.PKG, "csrc")
    for name in ("attn.cu", "attn.cuh", "attn_rows.cu", "gemv.cu", "heads.cu", "half_mma.cuh", "ops.cuh", "quant.cu", "quant.cuh"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        read = set(re.findall(r"__ldg\(\s*([\w.]+)", code))
        assert read <= ({"p.tile_ptr", "p.blk_kt", "p.g_w"} if name == "gemv.cu" else set()), (name, read)
        assert not re.search(r"const \w+\* __restrict__", code), name  # makes the same promise


def test_attention_layer_keeps_one_workspace_a_stream(L, monkeypatch):
    """Prompts of many lengths leave one buffer a stream, as large as the largest call's; the size
    does not fall as max_q grows, so what serves a call serves those of fewer query tokens."""
    from types import SimpleNamespace
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    sizes = [L.mq_kv_attention_workspace_bytes(32, 8, 128, q) for q in range(1, 100)]
    assert sizes == sorted(sizes) and 0 < sizes[0] < sizes[-1]
    now = ["a"]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[0])
    made = []

    def workspace(q, cache, max_q=1):
        made.append(torch.zeros(L.mq_kv_attention_workspace_bytes(q.shape[1], cache.heads, cache.D, max_q), dtype=torch.uint8))
        return made[-1]

    monkeypatch.setattr(mosaic, "kv_attention_workspace", workspace)
    cache, q = SimpleNamespace(heads=8, D=128), torch.zeros(1, 32, 128)
    layer = mosaic.AttentionLayer(SimpleNamespace(N=48 * 128), SimpleNamespace(K=32 * 128), 32, cache, None)
    for max_q in list(range(1, 60)) + [7, 4096, 1, 33]:
        ws = layer._workspace(q, max_q)
        assert ws.numel() >= L.mq_kv_attention_workspace_bytes(32, 8, 128, max_q)
    assert ws is layer._workspace(q, 5000) is layer._workspace(q, 1)
    assert sum(w.numel() for _, w in layer._ws.values()) == sizes[-1]
    now[0] = "b"
    assert layer._workspace(q, 9) is not ws and len(layer._ws) == 2
    now[0] = "a"
    assert layer._workspace(q, 2) is ws


def test_attention_layer_runs_on_the_device_of_its_tokens(monkeypatch):
    """With another device current, the whole step, prompts' projections among it, is launched with
    the tokens' device current, and the caller's device is current again after it."""
    from types import SimpleNamespace
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    at, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, at[0] = at[0], self.index

        def __exit__(self, *a):
            at[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch.cuda, "device", Device)

    class Layer(mosaic.AttentionLayer):
        def _project(self, layer, X):
            seen.append(at[0])
            raise KeyError  # nothing is launched here

    layer = Layer(SimpleNamespace(N=48 * 128), SimpleNamespace(K=32 * 128), 32, SimpleNamespace(heads=8, D=128), None)
    for dev in (1, 0):
        X = SimpleNamespace(shape=(20, 256), is_cuda=True, get_device=lambda: dev)
        with pytest.raises(KeyError):
            layer.step(X, None, None, None, None)
    assert seen == [1, 0] and at == [0]
    with pytest.raises(mosaic.MosaicError):
        layer.step(torch.zeros(20, 256, dtype=torch.bfloat16), None, None, None, None)


def test_the_library_is_built_without_the_extension(tmp_path, monkeypatch):
    """The C library comes first and needs nvcc alone; the timeline's needs no extension at all; an
    extension for another PyTorch is not taken for the running one's."""
    ran = []

    def call(cmd):
        ran.append(cmd[0])
        if cmd[0] != "nvcc":
            raise FileNotFoundError(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    real = build.marshal_path()
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "LIB_TIMELINE", str(tmp_path / "timeline.so"))
    monkeypatch.setattr(build.subprocess, "check_call", call)
    monkeypatch.delenv("NVCC", raising=False)
    monkeypatch.delenv("CXX", raising=False)
    with pytest.raises(FileNotFoundError):
        build.build()
    assert ran == ["nvcc", "g++"] and (tmp_path / "lib.so").exists() and not build.stale(build.LIB)
    assert build.build(timeline=True) == build.LIB_TIMELINE and ran == ["nvcc", "g++", "nvcc"]
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.1")
    assert os.path.basename(build.marshal_path()) != os.path.basename(real)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    pages = torch.zeros(2, 2, 1, 1152, dtype=torch.uint8)
    with pytest.raises(mosaic.MosaicError):
        mosaic.KVCache(pages)                              # a CPU tensor
    with pytest.raises(mosaic.MosaicError):
        mosaic.KVCache(pages.float())
    with pytest.raises(mosaic.MosaicError):
        mosaic.KVCache.alloc(2, 24, 2, 64, "cpu")
    x = torch.zeros(2, 2, 64)
    with pytest.raises(mosaic.MosaicError):                # fp32
        mosaic.mq_qk_norm_rope(x, None, x, None)
    y = x.to(torch.bfloat16)
    with pytest.raises(mosaic.MosaicError):                # two types
        mosaic.mq_qk_norm_rope(y, None, x.to(torch.float16), None)
    with pytest.raises(mosaic.MosaicError):                # a CPU tensor
        mosaic.mq_qk_norm_rope(y, None, y, None)
