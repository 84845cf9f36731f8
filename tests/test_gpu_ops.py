"""The operators of include/mosaic_ops.h on the GPU against plain 64-bit references: odd
sizes, strides, pages, ragged lengths, empty rows, NaN in places that no row sees, both
types, captured graphs, other streams, and a decoder layer's attention half run through
all of them. Quantized results are compared bit for bit with the CPU oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
import ops_ref as ref
import synth
from gpu_path import to_dev

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def mosaic():
    from bit_quantized_gemm_zipperengine_b200 import mosaic as m
    return m


@pytest.fixture(autouse=True)
def no_device_error(request):
    yield
    from bit_quantized_gemm_zipperengine_b200 import mosaic
    assert mosaic.mq_get_error() == 0


def within(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound)[bad].max()):.2f} x "
                           f"the bound, first at {torch.nonzero(bad)[0].tolist()}")


# ------------------------------------------------------------------------------ mq_gemv
def gemv_bound(x, W, y, g, dtype, K):
    """One rounding of the result, and the fp32 sum: K/16 accumulations of 16-element products
    (a tensor-core accumulation may truncate: 2^-23 of the running magnitude each), with 64
    more steps of 2^-24 for the sums between warps and the scale."""
    mag = (x.double().abs() @ W.abs().t()) * abs(g)
    e = (K / 8 + 64) * 2.0 ** -24 * mag
    return ref.rounding(y.abs() + e, dtype) + e


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K,budget", [(64, 64, 0), (64, 64, 1), (192, 320, 7), (128, 4096, 40), (576, 192, 27),
                                        (1024, 1088, 100), (256, 14336, 300)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gemv(M, N, K, budget, dtype, dev, mosaic):
    base, packed = ref.random_weight(N, K, budget, 11 * N + K, dev)
    gen = torch.Generator().manual_seed(M)
    hot = 1 + 29 * (torch.rand(K, generator=gen) < 0.02)
    x = (torch.randn(M, K, generator=gen) * hot * 0.1).to(dtype).to(dev)
    y = torch.full((M, N), math.nan, dtype=dtype, device=dev)
    mosaic.mq_gemv(x, mosaic.Weight(base, packed), y)
    W, g = ref.dense_weight(base, packed), float(base["gscale"])
    want = x.double() @ W.t() * g
    within(y, want, gemv_bound(x, W, want, g, dtype, K), f"M={M} {N}x{K}")


@pytest.mark.parametrize("mode", ["base", "residual"])
def test_gemv_parts_strides_flags(mode, dev, mosaic):
    N, K, M = 320, 704, 5
    base, packed = ref.random_weight(N, K, 20, 5, dev)
    big = torch.randn(M, K + 264, generator=torch.Generator().manual_seed(1)).to(BF).to(dev)
    x = big[:, 8:8 + K]
    out = torch.full((M, N + 7), 9.0, dtype=BF, device=dev)
    y = out[:, 3:3 + N]
    w = mosaic.Weight(base, packed)
    flag = mosaic.MQ_GEMM_BASE_ONLY if mode == "base" else mosaic.MQ_GEMM_RESIDUAL_ONLY
    mosaic.mq_gemv(x, w, y, flag | mosaic.MQ_GEMM_WEIGHTS_READY)
    W, g = ref.dense_weight(base, packed, mode), float(base["gscale"])
    want = x.double() @ W.t() * g
    within(y, want, gemv_bound(x, W, want, g, BF, K), mode)
    assert (out[:, :3] == 9).all() and (out[:, 3 + N:] == 9).all()
    first = y.clone()
    for _ in range(3):
        mosaic.mq_gemv(x, w, y, flag)
        assert torch.equal(first, y)


def test_gemv_bad_block_indices_are_reported_and_left_out(dev, mosaic):
    """Ranges past the packed store and columns past K meet the kernel's own checks."""
    N, K, M = 192, 320, 3
    base, packed = ref.random_weight(N, K, 7, 5, dev)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(9)).to(BF).to(dev)
    good = torch.empty(M, N, dtype=BF, device=dev)
    mosaic.mq_gemv(x, mosaic.Weight(base, packed), good)
    for field, at, bad in (("tile_ptr", 3, 2 ** 31 - 1), ("tile_ptr", 2, -5), ("blk_kt", 6, K // 64), ("blk_kt", 6, -1),
                           ("blk_kt", 6, 2 ** 31 - 1)):
        p = dict(packed)
        p[field] = packed[field].clone()
        p[field][at] = bad
        y = torch.empty_like(good)
        mosaic.mq_gemv(x, mosaic.Weight(base, p), y)
        assert mosaic.mq_get_error() == 1, (field, bad)
        assert torch.isfinite(y).all() and torch.equal(y[:, :64], good[:, :64])


@pytest.mark.parametrize("big", [1e-30, 1e30])
def test_gemv_far_magnitudes(big, dev, mosaic):
    """bf16 activations far outside fp16's range, and rows of very different size."""
    N, K, M = 128, 512, 4
    base, packed = ref.random_weight(N, K, 5, 8, dev)
    base["gscale"].fill_(2.0 ** -20)
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(2)) * torch.tensor([[big], [1.0], [0.0], [big * 7]])).to(BF).to(dev)
    y = torch.full((M, N), math.nan, dtype=BF, device=dev)
    mosaic.mq_gemv(x, mosaic.Weight(base, packed), y)
    W = ref.dense_weight(base, packed)
    want = x.double() @ W.t() * 2.0 ** -20
    within(y, want, gemv_bound(x, W, want, 2.0 ** -20, BF, K))


@pytest.mark.parametrize("big,g", [(1e36, 2.0 ** -20), (2.0 ** 125, 2.0 ** -36), (1e-37, 2.0 ** -10), (1e-38, 2.0 ** 30)])
def test_gemv_magnitudes_at_the_ends_of_bf16(big, g, dev, mosaic):
    """Activations near bf16's largest and smallest values, whose products' sums pass fp32's range
    before the tensor scale and lie inside it after."""
    N, K, M = 128, 512, 3
    base, packed = ref.random_weight(N, K, 5, 8, dev)
    base["gscale"].fill_(g)
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(2)).double() * torch.tensor([[big], [1.0], [big / 64]])).to(BF).to(dev)
    W = ref.dense_weight(base, packed)
    want = x.double() @ W.t() * g
    assert torch.isfinite(x).all() and want.abs().max() < torch.finfo(BF).max
    y = torch.full((M, N), math.nan, dtype=BF, device=dev)
    mosaic.mq_gemv(x, mosaic.Weight(base, packed), y)
    within(y, want, gemv_bound(x, W, want, g, BF, K))


def test_gemv_graphs_streams_and_workspaces(dev, mosaic):
    """A captured call replayed with other activations, calls on two streams at once, and a
    workspace of the caller's that an earlier call left full."""
    N, K, M = 512, 1024, 3
    base, packed = ref.random_weight(N, K, 20, 5, dev)
    w = mosaic.Weight(base, packed)
    W, g = ref.dense_weight(base, packed), float(base["gscale"])
    gen = torch.Generator().manual_seed(4)
    x, y = torch.randn(M, K, generator=gen).to(BF).to(dev), torch.empty(M, N, dtype=BF, device=dev)
    mosaic.mq_gemv(x, w, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mosaic.mq_gemv(x, w, y)
    for scale in (1.0, 1e-20, 300.0):
        x.copy_((scale * torch.randn(M, K, generator=gen)).to(BF))
        graph.replay()
        want = x.double() @ W.t() * g
        within(y, want, gemv_bound(x, W, want, g, BF, K))
    xs = [torch.randn(m, K, generator=gen).to(BF).to(dev) for m in (1, 16)]
    ys = [torch.empty(t.shape[0], N, dtype=BF, device=dev) for t in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, o, s in zip(xs, ys, streams):
            mosaic.mq_gemv(t, w, o, stream=s)
    torch.cuda.synchronize()
    ws = torch.full((mosaic.lib().mq_gemv_workspace_bytes(16, K),), 0x7F, dtype=torch.uint8, device=dev)
    for t, o in zip(xs, ys):
        want = t.double() @ W.t() * g
        within(o, want, gemv_bound(t, W, want, g, BF, K))
        again = torch.empty_like(o)
        mosaic.mq_gemv(t, w, again, ws=ws)
        assert torch.equal(o, again)


def test_gemv_reads_what_the_kernel_before_it_writes(dev, mosaic):
    """Activations, and operands of attention, written over and over by the launch just before:
    every call sees its own, not the call's before it."""
    N, K, M, n = 256, 1024, 8, 24
    base, packed = ref.random_weight(N, K, 9, 5, dev)
    w = mosaic.Weight(base, packed)
    gen = torch.Generator().manual_seed(7)
    src = torch.randn(n, M, K // 128, 128, generator=gen).to(BF).to(dev)
    x, ys = torch.empty(M, K // 128, 128, dtype=BF, device=dev), torch.empty(n, M, N, dtype=BF, device=dev)
    pages, ks, vs = ref.random_cache(4, 16, K // 128, 128, 3, dev)
    cache = mosaic.KVCache(pages, ks, vs)
    slots = torch.arange(M, device=dev)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.full((1,), M, dtype=torch.int32, device=dev)
    cu = torch.tensor([0, M], dtype=torch.int32, device=dev)
    os_, ws = torch.empty(n, M, K // 128, 128, dtype=BF, device=dev), mosaic.kv_attention_workspace(x, cache, M)

    def chain(i):
        mosaic.mq_qk_norm_rope(src[i], None, x, None)  # without norm and rotation: a copy
        mosaic.mq_gemv(x.view(M, K), w, ys[i])
        mosaic.mq_kv_append(x, x, slots, cache)
        mosaic.mq_kv_attention(x, cache, table, lens, os_[i], 0.09, cu, M, ws=ws)

    for i in range(n):
        chain(i)
        torch.cuda.synchronize()
    want = ys.clone(), os_.clone()
    ys.zero_(), os_.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            chain(i)
    for _ in range(10):
        graph.replay()
    assert torch.equal(ys, want[0]) and torch.equal(os_, want[1])


def test_gemv_on_a_prepared_layer(dev, mosaic):
    """The buffers that the layer's own preparation wrote, next to mq_gemm on the same weight."""
    L = synth.layer("tiny")
    N, K = L["N"], L["K"]
    budget = synth.budget_blocks(N, K, 0.10)
    layer = mosaic.Layer(N, K, budget, dev)
    layer.prepare_path(to_dev(L["W"], dev), to_dev(L["Xcal"], dev))
    X = to_dev(L["X"], dev)
    y = layer.forward_16bit(X)
    wq = oracle.quantize_weight(L["W"])
    sel = layer.sel[:budget].cpu().numpy()
    deq = oracle.nvfp4_dequantize(wq["codes"], wq["sf"], wq["g"]).astype(np.float64)
    res = oracle.nvfp4_dequantize(wq["r_codes"], wq["r_sf"], wq["g"]).astype(np.float64)
    mask = np.kron(oracle.block_mask(sel, N, K), np.ones((64, 64)))
    W = torch.from_numpy(deq + res * mask).to(dev)
    want = X.double() @ W.t()
    # the oracle's dequantized values carry one fp32 rounding each (2^-24)
    within(y, want, gemv_bound(X, W, want, 1.0, BF, K) + 2.0 ** -24 * (X.double().abs() @ W.abs().t()))


# ---------------------------------------------------------------------- norms and rotation
def rope_inputs(T, Hq, Hk, D, dtype, seed, dev, far=131072, theta=1e6, rot=None):
    gen = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(T, Hq + 2 * Hk, D, generator=gen)).to(dtype).to(dev)
    w = [(1 + 0.3 * torch.randn(D, generator=gen)).to(dtype).to(dev) for _ in range(2)]
    pos = torch.randint(0, far, (T,), generator=gen).to(dev)
    rot = D if rot is None else rot
    freq = (theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))).to(dev)
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], w, pos, freq


def rope_bound(want, mag, dtype):
    """The rounding, and fp32: 16 steps of 2^-24 for the sum of squares and its root, four
    for the products, 2^-21 for the angle's fp32 fraction (2^-24 of a turn) and its sine."""
    return ref.rounding(want, dtype) + 2.0 ** -19 * mag


@pytest.mark.parametrize("T,Hq,Hk,D,rot,norm,inter", [
    (1, 1, 1, 64, 64, True, False), (3, 5, 1, 128, 128, True, False), (17, 32, 8, 128, 64, True, True),
    (5, 7, 7, 256, 256, False, False), (2, 64, 8, 128, 128, False, True), (9, 3, 3, 64, 16, True, False),
    (4, 6, 2, 128, 96, False, False), (33, 4, 2, 256, 32, True, True), (6, 4, 4, 128, 0, True, False)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_norm_rope(T, Hq, Hk, D, rot, norm, inter, dtype, dev, mosaic):
    q, k, _, w, pos, freq = rope_inputs(T, Hq, Hk, D, dtype, T * D + rot, dev, rot=rot)
    wq, wk = w if norm else (None, None)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty(Hk, T, D, dtype=dtype, device=dev).transpose(0, 1)
    want = [ref.norm_rope(x, u, 1e-6, pos, freq, rot, inter) for x, u in ((q, wq), (k, wk))]
    mosaic.mq_qk_norm_rope(q, k, qo, ko, pos, freq if rot else None, wq, wk, 1e-6, inter)
    for got, (y, mag) in zip((qo, ko), want):
        within(got, y, rope_bound(y, mag, dtype))
    # in place, one side at a time: the same bits
    mosaic.mq_qk_norm_rope(q, None, q, None, pos, freq if rot else None, wq, None, 1e-6, inter)
    mosaic.mq_qk_norm_rope(None, k, None, k, pos, freq if rot else None, None, wk, 1e-6, inter)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("T,Hq", [(5, 3), (1, 4), (6, 1)])
def test_norm_rope_output_layouts(T, Hq, dev, mosaic):
    """Tokens inside heads, heads inside tokens, gaps, and axes of one element with stride 0."""
    D = 64
    q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(4)).to(BF).to(dev)
    pos, freq = torch.arange(T, device=dev), (1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).to(dev)
    want = torch.empty_like(q)
    mosaic.mq_qk_norm_rope(q, None, want, None, pos, freq)
    mem = torch.empty(T * Hq * D * 4, dtype=BF, device=dev)
    for st, sh in ((D, T * D), (Hq * D, D), (Hq * (D + 8) + 16, D + 8), (D + 8, T * (D + 8)), (0 if T == 1 else Hq * D, 0 if Hq == 1 else D)):
        o = mem.as_strided((T, Hq, D), (st, sh, 1))
        mosaic.mq_qk_norm_rope(q, None, o, None, pos, freq)
        assert torch.equal(o, want), (st, sh)


def test_binding_arguments_that_are_no_numbers(dev, mosaic):
    """A flag or truth value that cannot be taken is an error of the call, and nothing is launched."""
    q = torch.ones(2, 2, 64, dtype=BF, device=dev)
    out = torch.zeros_like(q)
    base, packed = ref.random_weight(64, 64, 0, 1, dev)
    x, y = torch.ones(1, 64, dtype=BF, device=dev), torch.zeros(1, 64, dtype=BF, device=dev)
    at = mosaic.mq_launch_count()
    with pytest.raises(RuntimeError, match="ambiguous"):
        mosaic.mq_qk_norm_rope(q, None, out, None, interleaved=torch.zeros(2))
    with pytest.raises(TypeError):
        mosaic.mq_qk_norm_rope(q, None, out, None, eps="small")
    for flags in (2 ** 32, 2 ** 33 + 4, -2 ** 40):
        with pytest.raises(mosaic.MosaicError):
            mosaic.mq_gemv(x, mosaic.Weight(base, packed), y, flags)
    with pytest.raises(TypeError):
        mosaic.mq_gemv(x, mosaic.Weight(base, packed), y, "base")
    torch.cuda.synchronize()
    assert mosaic.mq_launch_count() == at and (out == 0).all() and (y == 0).all()


def test_rope_far_positions_and_zero_rows(dev, mosaic):
    q, k, _, w, pos, freq = rope_inputs(8, 2, 1, 128, HF, 3, dev)
    pos = torch.tensor([0, 1, -5, 2 ** 20, 2 ** 31, 2 ** 40, -(2 ** 33), 7], device=dev)
    q[3] = 0
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    mosaic.mq_qk_norm_rope(q, k, qo, ko, pos, freq, w[0], w[1], 1e-6)
    for got, x, u in ((qo, q, w[0]), (ko, k, w[1])):
        y, mag = ref.norm_rope(x, u, 1e-6, pos, freq, 128, False)
        # the angle itself is one fp64 product: 2^-53 of it is unknown to both sides
        within(got, y, rope_bound(y, mag, HF) + 2.0 ** -52 * pos.abs().double()[:, None, None] * mag)
    assert (qo[3] == 0).all()


# ----------------------------------------------------------------------------- the cache
def oracle_rows(x, g):
    """(codes, scales) by the CPU oracle of rows x [T][H][D] with tensor scales g [H]."""
    T, H, D = x.shape
    gs = np.ones(T * H, np.float32) if g is None else np.tile(g.cpu().numpy(), T)
    if T * H == 1:  # one row: the oracle takes a scalar
        gs = gs[0]
    r = oracle.nvfp4_quantize(x.float().cpu().numpy().reshape(T * H, D), gs)
    return r["codes"].reshape(T, H, D // 2), r["sf"].reshape(T, H, D // 16), r["deq"].reshape(T, H, D)


@pytest.mark.parametrize("T,H,D,P,pages", [(1, 1, 64, 16, 1), (1, 8, 128, 64, 3), (37, 3, 128, 16, 5), (100, 2, 64, 32, 4),
                                           (256, 8, 128, 128, 4)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scales", [True, False])
def test_append_and_read(T, H, D, P, pages, dtype, scales, dev, mosaic):
    gen = torch.Generator().manual_seed(T + D)
    kv = torch.randn(T, 2 * H + 1, D, generator=gen)
    kv[0, 0, :16] = 0                       # a group of zeros
    kv[-1, H, :16] = 3000.0                 # one beyond the largest value
    kv[0, :, 16:32] *= 1e-5                 # one whose scale underflows
    kv = kv.to(dtype).to(dev)
    k, v = kv[:, :H], kv[:, H:2 * H]
    bytes_, ks, vs = ref.random_cache(pages, P, H, D, 1, dev, scales)
    before = bytes_.clone()
    cache = mosaic.KVCache(bytes_, ks, vs)
    slots = torch.randperm(pages * P, generator=gen)[:T].to(dev)
    mosaic.mq_kv_append(k, v, slots, cache)
    ko, vo = torch.empty(T, H, D, dtype=dtype, device=dev), torch.empty(T, H, D, dtype=dtype, device=dev)
    mosaic.mq_kv_read(cache, slots, ko, vo)
    want = before.cpu().numpy()
    maps = [m.numpy() for m in ref.record_maps(D, "cpu")]
    s = slots.cpu().numpy()
    for x, g, cm, sm, got in ((k, ks, maps[0], maps[2], ko), (v, vs, maps[1], maps[3], vo)):
        codes, sf, deq = oracle_rows(x, g)
        for t in range(T):
            page, rec, i = s[t] // P, s[t] % P // 16, s[t] % 16
            want[page, :, rec][:, cm[i, ::2]] = codes[t]
            want[page, :, rec][:, sm[i, ::16]] = sf[t]
        assert torch.equal(got.cpu(), torch.from_numpy(deq).to(dtype))
    assert np.array_equal(bytes_.cpu().numpy(), want)  # and nothing beside them


def test_append_skips_and_reports(dev, mosaic):
    H, D, P = 2, 64, 16
    bytes_, ks, vs = ref.random_cache(2, P, H, D, 4, dev)
    cache, before = mosaic.KVCache(bytes_, ks, vs), bytes_.clone()
    k = torch.randn(4, H, D, device=dev).to(BF)
    slots = torch.tensor([-1, -2 ** 40, -1, -7], device=dev)
    mosaic.mq_kv_append(k, k, slots, cache)
    ko, vo = torch.full_like(k, 5.0), torch.full_like(k, 6.0)
    mosaic.mq_kv_read(cache, slots, ko, vo)
    assert torch.equal(bytes_, before) and (ko == 5).all() and (vo == 6).all() and mosaic.mq_get_error() == 0
    # past the cache: left out by the kernels' own checks, and reported
    for call in (lambda s: mosaic.mq_kv_append(k, k, s, cache), lambda s: mosaic.mq_kv_read(cache, s, ko, vo)):
        call(torch.tensor([-1, 2 * P, -1, 2 ** 50], device=dev))
        assert mosaic.mq_get_error() == 1
        assert torch.equal(bytes_, before) and (ko == 5).all() and (vo == 6).all()


@pytest.mark.parametrize("T,Hq,H,D,rot,norm,inter", [(1, 8, 2, 128, 128, True, False), (19, 3, 3, 64, 32, False, True),
                                                     (64, 64, 8, 128, 128, True, False)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_qkv_append_is_the_two_calls(T, Hq, H, D, rot, norm, inter, dtype, dev, mosaic):
    q, k, v, w, pos, freq = rope_inputs(T, Hq, H, D, dtype, T, dev, rot=rot)
    wq, wk = w if norm else (None, None)
    bytes_, ks, vs = ref.random_cache(8, 16, H, D, 2, dev)
    slots = torch.randperm(128, generator=torch.Generator().manual_seed(T))[:T].to(dev)
    slots[T // 2] = -1 if T > 1 else slots[0]
    a, b, c = (mosaic.KVCache(bytes_.clone(), ks, vs) for _ in range(3))
    qo, ko, q2, k2 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k)
    mosaic.mq_qk_norm_rope(q, k, qo, ko, pos, freq, wq, wk, 1e-6, inter)
    mosaic.mq_kv_append(ko, v, slots, a)
    mosaic.mq_qkv_append(q, k, v, q2, slots, b, pos, freq, wq, wk, 1e-6, inter, k_out=k2)
    assert torch.equal(qo, q2) and torch.equal(ko, k2) and torch.equal(a.pages, b.pages)
    mosaic.mq_qkv_append(q, k, v, q, slots, c, pos, freq, wq, wk, 1e-6, inter)  # in place, keys kept in the cache alone
    assert torch.equal(qo, q) and torch.equal(a.pages, c.pages)


# ------------------------------------------------------------------------------ attention
def attn_inputs(lens, nqs, Hq, H, D, P, dtype, seed, dev, extra_pages=2, qmul=1.0):
    gen = torch.Generator().manual_seed(seed)
    per = max(1, -(-max(lens) // P))
    need = [-(-n // P) for n in lens]
    pages, ks, vs = ref.random_cache(sum(need) + extra_pages, P, H, D, seed + 1, dev)
    ids = torch.randperm(sum(need) + extra_pages, generator=gen)
    table = torch.full((len(lens), per), -1, dtype=torch.int32)  # -1 behind each sequence's pages
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n].int()
        at += n
    ref.poison(pages, table, lens)
    T = sum(nqs)
    q = (qmul * torch.randn(T + 2, Hq + 1, D, generator=gen)).to(dtype).to(dev)[:T, :Hq]
    cu = torch.tensor([0] + list(np.cumsum(nqs)), dtype=torch.int32, device=dev)
    return q, pages, ks, vs, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), cu


def attn_bounds(out, lse, mass, smax, vmax, dtype, lens):
    """Scores: D products of an exact fp16 pair in fp32 and one scale: 2^-20 (1 + max |s|)
    covers them and exp2's 2^-22. The softmax weights enter the second product in fp16 (half
    a step is 2^-11; below 2^-21 of the row's largest the step is absolute, 2^-32 of it a
    token), summed in fp32 (n / 8 steps of 2^-24 and 64 for the joins)."""
    n = max(lens)
    d = 2.0 ** -20 * (1 + smax)
    e = mass * (2.0 ** -11 + (n / 8 + 64) * 2.0 ** -24 + 2 * d[..., None]) + n * 2.0 ** -32 * vmax[..., None]
    return ref.rounding(out.abs() + e, dtype) + e, d + (n / 8 + 64) * 2.0 ** -24 + 2.0 ** -23 * lse.abs().nan_to_num(posinf=0.0)


def run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max_q, scale, window, dtype, use_cu=True, ws=None):
    T, Hq, D = q.shape
    cache = mosaic.KVCache(pages, ks, vs)
    out = torch.full((T, Hq + 3, D), 77.0, dtype=dtype, device=q.device)
    o = out[:, 1:1 + Hq]
    lse = torch.full((T, Hq), 77.0, device=q.device)
    ws = mosaic.kv_attention_workspace(q, cache, max_q) if ws is None else ws
    mosaic.mq_kv_attention(q, cache, table, kv_len, o, scale, cu if use_cu else None, max_q, window, lse, ws)
    assert (out[:, 0] == 77).all() and (out[:, 1 + Hq:] == 77).all()
    return o, lse


CASES = [
    # lens, query tokens, Hq, H, D, P, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [1], 8, 8, 128, 64, 0),
    ([15, 16, 17, 33], [1] * 4, 8, 2, 128, 16, 0),
    ([127, 128, 129, 1, 255], [1] * 5, 6, 1, 128, 32, 0),
    ([0, 5, 300], [1] * 3, 12, 4, 64, 64, 0),
    ([700, 3], [1] * 2, 64, 8, 128, 128, 0),
    ([515, 64], [1] * 2, 20, 1, 128, 16, 0),          # 20 query heads on one
    ([400, 90, 7], [1] * 3, 4, 4, 128, 16, 33),       # a window
    ([400, 129], [1] * 2, 8, 1, 64, 64, 1),           # a window of one
    ([40, 3, 200], [5, 3, 1], 8, 2, 128, 32, 0),      # several query tokens
    ([2, 40], [5, 2], 8, 8, 128, 16, 0),              # more query tokens than cached: rows that see nothing
    ([0, 0], [2, 1], 4, 2, 64, 16, 0),
    ([300, 70], [70, 0], 6, 2, 128, 64, 0),           # a whole prompt; a sequence without query tokens
    ([513], [200], 4, 1, 64, 32, 100),
    ([260, 31], [130, 31], 8, 1, 128, 16, 17),
    ([1030] + [9] * 40, [1] * 41, 8, 2, 128, 16, 0),  # one long among many short
    ([5000], [1], 8, 1, 128, 64, 0),                  # cut into many pieces
    ([3001, 2999], [3, 4], 16, 2, 64, 16, 0),
    ([97, 500, 48, 49], [1] * 4, 8, 4, 128, 48, 0),   # pages that are no power of two
    ([(7 * i) % 90 for i in range(300)], [1] * 300, 8, 2, 64, 16, 0),             # more sequences than threads of a CTA
    ([40 + (11 * i) % 200 for i in range(140)], [i % 4 for i in range(140)], 4, 1, 128, 32, 50),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention(case, dtype, dev, mosaic):
    lens, nqs, Hq, H, D, P, window = CASES[case]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, Hq, H, D, P, dtype, case, dev)
    scale = D ** -0.5
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, scale, window)
    one = all(n == 1 for n in nqs)
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max(nqs), scale, window, dtype, not one)
    bo, bl = attn_bounds(*want, dtype, lens)
    within(o, want[0], bo, "out")
    dead = want[1] == -math.inf
    assert (lse[dead] == -math.inf).all() and (o[dead] == 0).all()
    within(lse[~dead], want[1][~dead], bl[~dead], "lse")
    # the same bits again; a too small expectation of max_q only picks another kernel
    o2, lse2 = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max(nqs), scale, window, dtype, not one)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if one:
        o3, _ = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 1, scale, window, dtype, True)
        assert torch.equal(o, o3)
    else:
        o3, _ = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 1, scale, window, dtype, True)
        within(o3, want[0], bo, "out, max_q = 1")


ROWS = [
    # many query rows a cache head: lens, query tokens, Hq, H, P, window
    ([700, 301], [300, 301], 64, 16, 64, 0),
    ([900, 1], [800, 1], 32, 32, 16, 0),                  # a head of its own for each query head
    ([256, 9, 40], [256, 0, 77], 80, 16, 48, 50),         # a window; more query tokens than cached
    ([3000, 64, 64], [200, 64, 65], 96, 16, 128, 0),      # behind a prefix
    ([640, 700], [128, 600], 64, 16, 32, 129),
    ([0, 500], [130, 400], 40, 20, 16, 0),                # rows that see nothing
    ([64, 65, 63, 129], [64, 65, 63, 129], 128, 32, 64, 1),
]


@pytest.mark.parametrize("case", range(len(ROWS)))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_many_rows(case, dtype, dev, mosaic):
    lens, nqs, Hq, H, P, window = ROWS[case]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, Hq, H, 128, P, dtype, 70 + case, dev, qmul=1.0 + case)
    scale = (-1) ** case * 128 ** -0.5
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, scale, window)
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max(nqs), scale, window, dtype)
    bo, bl = attn_bounds(*want, dtype, lens)
    within(o, want[0], bo, "out")
    dead = want[1] == -math.inf
    assert (lse[dead] == -math.inf).all() and (o[dead] == 0).all()
    within(lse[~dead], want[1][~dead], bl[~dead], "lse")
    o2, lse2 = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max(nqs), scale, window, dtype)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


MIXED = [
    # prompts beside single tokens and drafts, by two kernels: (query tokens, cached), Hq, H, P, window
    ([(1, 700), (300, 301), (1, 5), (0, 40), (200, 200), (1, 0), (7, 90)], 64, 16, 16, 0),
    ([(300, 300) if i in (0, 33, 69) else (1, (37 * i) % 150) for i in range(70)], 32, 16, 32, 0),
    ([(260, 100 + i) if i in (5, 140) else (i % 3, (11 * i) % 90) for i in range(150)], 64, 16, 16, 60),
    ([(64, 20000), (300, 300), (1, 129)], 64, 16, 64, 0),       # many rows, and too long for one CTA each
    ([(1, 3000), (130, 40), (2, 1), (150, 1000)], 64, 16, 48, 0),  # more query tokens than cached
    ([(31, 64), (32, 64), (33, 64), (200, 64)], 128, 32, 64, 0),   # beside the least rows
]


@pytest.mark.parametrize("case", range(len(MIXED)))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_mixed(case, dtype, dev, mosaic):
    seqs, Hq, H, P, window = MIXED[case]
    nqs, lens = [s[0] for s in seqs], [s[1] for s in seqs]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, Hq, H, 128, P, dtype, 170 + case, dev)
    scale = (-1) ** case * 128 ** -0.5
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, scale, window)
    bo, bl = attn_bounds(*want, dtype, lens)
    dead = want[1] == -math.inf
    q = torch.cat((q, q[:5]))  # rows of no sequence
    first = None
    for max_q in (max(nqs), 1, 10 * max(nqs)):
        at = mosaic.mq_launch_count()
        o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max_q, scale, window, dtype)
        if max_q == max(nqs):
            assert mosaic.mq_launch_count() == at + 2
            first = o.clone(), lse.clone()
        assert (o[-5:] == 77).all() and (lse[-5:] == 77).all()
        o, lse = o[:-5], lse[:-5]
        within(o, want[0], bo, "out")
        assert (lse[dead] == -math.inf).all() and (o[dead] == 0).all()
        within(lse[~dead], want[1][~dead], bl[~dead], "lse")
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max(nqs), scale, window, dtype)
    assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    # a page that is not there, and a length past the table, in both kinds: the others as they were
    for b in range(min(2, len(lens))):
        if lens[b] > P:
            t = table.clone()
            t[b, 1] = pages.shape[0]
            o, _ = run_attn(mosaic, q, pages, ks, vs, t, kv_len, cu, max(nqs), scale, window, dtype)
            assert mosaic.mq_get_error() == 1
            rest = torch.ones(sum(nqs), dtype=torch.bool, device=dev)
            rest[int(cu[b]):int(cu[b + 1])] = False
            within(o[:-5][rest], want[0][rest], bo[rest])


@pytest.mark.parametrize("nq,B,Hq,H,long,window", [(8, 16, 64, 8, 9000, 0), (1, 130, 64, 1, 12000, 0), (13, 20, 32, 8, 700, 300)])
def test_attention_as_many_tokens_each_and_ragged_lengths(nq, B, Hq, H, long, window, dev, mosaic):
    """As many query tokens each, rows enough for the kernel of many rows, one context far longer."""
    lens = [long if i == B // 2 else (37 * i) % 210 for i in range(B)]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, [nq] * B, Hq, H, 128, 16, BF, 200 + nq, dev)
    want = ref.attention(q, pages, ks, vs, table, lens, [nq] * B, 0.09, window)
    bo, bl = attn_bounds(*want, BF, lens)
    dead = want[1] == -math.inf
    at = mosaic.mq_launch_count()
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, nq, 0.09, window, BF, nq > 1)
    assert mosaic.mq_launch_count() == at + 2
    within(o, want[0], bo, "out")
    assert (lse[dead] == -math.inf).all() and (o[dead] == 0).all()
    within(lse[~dead], want[1][~dead], bl[~dead], "lse")
    again = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, nq, 0.09, window, BF, nq > 1)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_attention_mixed_in_graphs(dev, mosaic):
    """A captured chain of calls, each the next one's queries, replayed with other rows and lengths:
    which kernel has which sequence changes, and the next call sees what both wrote."""
    B, T, Hq, H, P, most = 4, 400, 64, 16, 32, 512
    q, pages, ks, vs, table, kv_len, cu = attn_inputs([most] * B, [100] * B, Hq, H, 128, P, BF, 190, dev)
    q = q.contiguous()
    cache = mosaic.KVCache(pages, ks, vs)
    ws = mosaic.kv_attention_workspace(q, cache, T)
    outs = [torch.empty_like(q) for _ in range(3)]

    def chain(sync=False):
        x = q
        for o in outs:
            mosaic.mq_kv_attention(x, cache, table, kv_len, o, 0.09, cu, T, ws=ws)
            x = o
            if sync:
                torch.cuda.synchronize()

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for rows, lens in (([0, 300, 301, 302, 400], [300, 512, 1, 100]), ([0, 1, 2, 3, 400], [512, 0, 77, 397]),
                       ([0, 100, 200, 300, 400], [512, 100, 300, 101]), ([0, 0, 0, 0, 400], [1, 2, 3, 400]),
                       ([0, 400, 400, 400, 400], [64, 1, 1, 1]), ([0, 20, 40, 41, 60], [512, 500, 400, 300])):
        cu.copy_(torch.tensor(rows, dtype=torch.int32))
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        for o in outs:
            o.fill_(0.5)
        chain(sync=True)
        want = [o.clone() for o in outs]
        nqs = [b - a for a, b in zip(rows, rows[1:])]
        w = ref.attention(q[:rows[-1]], pages, ks, vs, table, lens, nqs, 0.09, 0)
        within(want[0][:rows[-1]], w[0], attn_bounds(*w, BF, lens)[0], str(rows))
        for o in outs:
            o.fill_(0.5)
        for _ in range(3):
            graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rows


def test_attention_many_rows_single_tokens(dev, mosaic):
    """One query token a sequence (no cu_q), 64 query heads on one."""
    lens = [(37 * i) % 290 for i in range(130)]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, [1] * 130, 64, 1, 128, 16, BF, 95, dev)
    want = ref.attention(q, pages, ks, vs, table, lens, [1] * 130, 0.09, 100)
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 1, 0.09, 100, BF, False)
    within(o, want[0], attn_bounds(*want, BF, lens)[0])
    assert (o[want[1] == -math.inf] == 0).all()


def test_attention_many_rows_in_graphs(dev, mosaic):
    """A captured prompt replayed with other lengths, between calls of the other kernel and a
    product that holds tensor memory too."""
    lens, nqs = [700, 640], [300, 301]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 64, 16, 128, 64, BF, 97, dev)
    cache = mosaic.KVCache(pages, ks, vs)
    out, small = torch.empty_like(q).contiguous(), torch.empty(2, 64, 128, dtype=BF, device=dev)
    ws = mosaic.kv_attention_workspace(q, cache, 301)
    layer = mosaic.Layer(256, 512, 3, dev)
    layer.prepare_path(to_dev(synth.weight(256, 512, 1, 2, 0.06, 40, 2, 8.0), dev), to_dev(synth.act(128, 512, 3, 4, 4, 5.0), dev))
    X = torch.randn(64, 512, generator=torch.Generator().manual_seed(1)).to(BF).to(dev)

    def call():
        y = layer.forward(X)
        mosaic.mq_kv_attention(q, cache, table, kv_len, out, 0.09, cu, 301, ws=ws)
        mosaic.mq_kv_attention(q[:2], cache, table, kv_len, small, 0.09, ws=ws)
        return y, layer.forward(X)

    y = call()[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = call()
    for now in (lens, [320, 301], [1, 640]):
        kv_len.copy_(torch.tensor(now, dtype=torch.int32))
        for _ in range(3):
            graph.replay()
        want = ref.attention(q, pages, ks, vs, table, now, nqs, 0.09, 0)
        within(out, want[0], attn_bounds(*want, BF, lens)[0], str(now))
        want = ref.attention(q[:2], pages, ks, vs, table, now, [1, 1], 0.09, 0)
        within(small, want[0], attn_bounds(*want, BF, lens)[0], str(now))
        assert torch.equal(ys[0], y) and torch.equal(ys[1], y)


def test_attention_many_rows_bad_pages_and_nan(dev, mosaic):
    """A page that is not there leaves its tokens out, as the same cache without them would; a
    NaN in a query stays in its row; rows of no sequence stay as they were."""
    lens, nqs, P = [640, 300], [400, 300], 64
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 64, 16, 128, P, BF, 91, dev)
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, 0.09, 0)
    bound = attn_bounds(*want, BF, lens)[0]
    q = torch.cat((q, q[:3]))
    q[7, 5, 100] = math.nan
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=dev)
    hit[7, 5] = True
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 400, 0.09, 0, BF)
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all() and (o[700:] == 77).all() and (lse[700:] == 77).all()
    ok = ~hit[:700]
    within(o[:700][ok], want[0][ok], bound[ok])
    for bad in (-1, pages.shape[0]):
        t = table.clone()
        t[0, 9] = bad  # the last 64 tokens of the first sequence
        o, lse = run_attn(mosaic, q, pages, ks, vs, t, kv_len, cu, 400, 0.09, 0, BF)
        assert mosaic.mq_get_error() == 1
        # rows in front of the page are unchanged; those behind it see what a window of none would
        within(o[:336][ok[:336]], want[0][:336][ok[:336]], bound[:336][ok[:336]])
        at576 = ref.attention(q[335:336], pages, ks, vs, table, [576], [1], 0.09, 0)
        q1 = q.clone()
        q1[336:400] = q[335]
        o, _ = run_attn(mosaic, q1, pages, ks, vs, t, kv_len, cu, 400, 0.09, 0, BF)
        assert mosaic.mq_get_error() == 1
        within(o[335:400], at576[0].expand(65, -1, -1), attn_bounds(*at576, BF, [576])[0].expand(65, -1, -1))
        within(o[400:700], want[0][400:], bound[400:], "the other sequence")


@pytest.mark.parametrize("qmul,scale", [(60.0, 0.5), (1e-3, 1.0), (1.0, 0.0), (4.0, -0.3)])
def test_attention_sharp_flat_and_odd_scales(qmul, scale, dev, mosaic):
    lens, nqs = [777, 64, 1], [2, 1, 1]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 8, 2, 128, 32, BF, 9, dev, qmul=qmul)
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, scale, 0)
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 2, scale, 0, BF)
    bo, bl = attn_bounds(*want, BF, lens)
    within(o, want[0], bo, "out")
    within(lse, want[1], bl, "lse")


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1])
def test_attention_huge_windows(window, dev, mosaic):
    """A window that holds every token, with more query tokens than cached ones, is no window."""
    lens, nqs = [2, 40, 0], [5, 2, 3]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 8, 2, 64, 16, BF, 12, dev)
    want = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 5, 0.125, 0, BF)
    got = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 5, 0.125, window, BF)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_query_beyond_fp16(dev, mosaic):
    """bf16 queries far above and below fp16's range, with a scale that brings the scores back."""
    lens, nqs = [300], [4]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 8, 2, 128, 32, BF, 10, dev)
    q = (q.float() * torch.tensor([1e20, 1.0, 1e-20, 1e24], device=dev)[:, None, None]).to(BF)
    for scale in (1e-21, 1e18):
        if scale > 1:
            q[0], q[3], q[1] = 0, 0, 0
        want = ref.attention(q, pages, ks, vs, table, lens, nqs, scale, 0)
        o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 4, scale, 0, BF)
        bo, bl = attn_bounds(*want, BF, lens)
        within(o, want[0], bo, "out")
        within(lse, want[1], bl, "lse")


@pytest.mark.parametrize("rows", [False, True])
def test_attention_smallest_queries(rows, dev, mosaic):
    """bf16 queries near the smallest normal value with a scale that brings the scores back, in
    both kernels: the scale of a row is not rounded to a subnormal on the way."""
    lens, nqs = ([700, 301], [300, 301]) if rows else ([300], [4])
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 64 if rows else 8, 16 if rows else 2, 128, 32, BF, 13, dev)
    q, ks = (q.float() * 2.0 ** -122).to(BF), ks * 2.0 ** -9
    scale = 2.0 ** 124
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, scale, 0)
    assert want[3].max() < 200
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, max(nqs), scale, 0, BF)
    bo, bl = attn_bounds(*want, BF, lens)
    within(o, want[0], bo, "out")
    within(lse, want[1], bl, "lse")


def test_attention_nan_queries(dev, mosaic):
    """A query row that holds a NaN gives NaN for itself, its lse too, and for no other row."""
    lens, nqs = [1500, 40, 0], [1, 3, 1]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 8, 2, 128, 16, BF, 22, dev)
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, 0.1, 0)
    bo, bl = attn_bounds(*want, BF, lens)
    q = q.contiguous()
    for t, h in ((0, 3), (2, 6), (4, 1)):
        q[t, h, 17] = math.nan
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 3, 0.1, 0, BF)
    hit = torch.zeros(o.shape[:2], dtype=torch.bool, device=dev)
    hit[0, 3] = hit[2, 6] = True  # the third sees nothing: zeros
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    within(o[~hit], want[0][~hit], bo[~hit], "the other rows")
    dead = want[1] == -math.inf
    assert (lse[dead] == -math.inf).all() and (o[dead] == 0).all()
    within(lse[~hit & ~dead], want[1][~hit & ~dead], bl[~hit & ~dead], "lse")


def test_attention_bad_indices_are_reported_and_left_out(dev, mosaic):
    """Bad pages, lengths and rows meet the kernels' own checks: their tokens are left out."""
    lens, nqs = [100, 40], [1, 1]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 8, 2, 128, 16, BF, 21, dev)
    good = ref.attention(q, pages, ks, vs, table, lens, nqs, 0.1, 0)
    bound = attn_bounds(*good, BF, lens)[0]
    for bad in (-1, pages.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        o, _ = run_attn(mosaic, q, pages, ks, vs, t, kv_len, cu, 1, 0.1, 0, BF)
        assert mosaic.mq_get_error() == 1
        assert torch.isfinite(o).all()
        within(o[1], good[0][1], bound[1], "the other sequence")
    for n in (-3, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        o, lse = run_attn(mosaic, q, pages, ks, vs, table, torch.tensor([n, 40], dtype=torch.int32, device=dev), cu, 1, 0.1, 0, BF)
        assert mosaic.mq_get_error() == 1
        assert (o[0] == 0).all() and (lse[0] == -math.inf).all()
        within(o[1], good[0][1], bound[1], "the other sequence")
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, torch.tensor([0, 1, 9], dtype=torch.int32, device=dev), 1, 0.1, 0, BF)
    assert mosaic.mq_get_error() == 1  # rows past T
    within(o[0], good[0][0], bound[0], "the first sequence")
    assert (o[1] == 77).all()


def without_pages(table, lens, P, bad):
    """Table and lengths of single-token sequences whose pages `bad` (b, i) are cut out: what is left
    when a page is not there (the order of a sequence's tokens does not matter to its last one)."""
    t, n = table.clone(), list(lens)
    for b in range(len(lens)):
        gone = {i for c, i in bad if c == b}
        keep = [i for i in range(-(-lens[b] // P)) if i not in gone]
        t[b, :len(keep)] = table[b, torch.tensor(keep, device=table.device, dtype=torch.long)]
        n[b] = lens[b] - sum(min(P, lens[b] - i * P) for i in gone)
    return t, n


@pytest.mark.parametrize("lens,Hq,H,D,P,bad", [
    ([100, 40], 8, 2, 128, 16, [(0, 2)]),
    ([100, 47], 8, 2, 64, 16, [(0, 0), (0, 1), (1, 2)]),         # a whole step, and a last page in part
    ([3000], 8, 2, 128, 48, [(0, 0), (0, 30), (0, 31), (0, 62)]),
    # about 20 steps of every warp: pages of the first 16, which are looked up together, and behind them
    ([140000], 16, 8, 64, 64, [(0, i) for i in (0, 1, 17, 31, 32, 33, 34, 35, 36, 37, 38, 39, 40, 700, 1331, 1332, 2000, 2186, 2187)]),
    ([140000], 16, 8, 64, 64, [(0, i) for i in range(5, 2188, 13)]),
])
def test_attention_missing_pages_are_left_out(lens, Hq, H, D, P, bad, dev, mosaic):
    """Single tokens whose sequences miss pages: the result of the tokens that are there."""
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, [1] * len(lens), Hq, H, D, P, BF, 23, dev)
    t2, n2 = without_pages(table, lens, P, bad)
    want = ref.attention(q, pages, ks, vs, t2, n2, [1] * len(lens), 0.1, 0)
    bo, bl = attn_bounds(*want, BF, lens)
    for name in (-1, pages.shape[0]):
        t = table.clone()
        for b, i in bad:
            t[b, i] = name
        o, lse = run_attn(mosaic, q, pages, ks, vs, t, kv_len, cu, 1, 0.1, 0, BF, False)
        assert mosaic.mq_get_error() == 1
        within(o, want[0], bo, "out")
        within(lse, want[1], bl, "lse")


@pytest.mark.parametrize("lens,nqs,Hq,H,D,window", [
    ([515, 64], [1, 1], 20, 1, 128, 0), ([3001, 40, 7], [5, 5, 5], 16, 4, 128, 0), ([900, 2, 300], [3, 3, 3], 16, 2, 64, 70),
    ([700, 61], [4, 6], 32, 8, 64, 0), ([1500, 30], [17, 1], 2, 2, 128, 0)])
def test_attention_tables_of_great_capacity(lens, nqs, Hq, H, D, window, dev, mosaic):
    """17 to 24 query rows, with tables as long as the sequences and with far longer ones: another
    tile of rows, the same attention; one workspace serves both."""
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, Hq, H, D, 16, BF, 240 + D + Hq, dev)
    want = ref.attention(q, pages, ks, vs, table, lens, nqs, 0.09, window)
    bo, bl = attn_bounds(*want, BF, lens)
    dead = want[1] == -math.inf
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    wide = torch.full((len(lens), -(-8 * 2 * sms * 128 // (16 * H * len(lens))) + 8), -1, dtype=torch.int32, device=dev)
    wide[:, :table.shape[1]] = table
    ws = mosaic.kv_attention_workspace(q, mosaic.KVCache(pages, ks, vs), max(nqs))
    for t in (table, wide, table):
        o, lse = run_attn(mosaic, q, pages, ks, vs, t, kv_len, cu, max(nqs), 0.09, window, BF, ws=ws)
        within(o, want[0], bo, "out")
        assert (lse[dead] == -math.inf).all() and (o[dead] == 0).all()
        within(lse[~dead], want[1][~dead], bl[~dead], "lse")


def test_attention_shapes_share_a_workspace(dev, mosaic):
    """Calls of different shapes take turns on one workspace, large enough for each: the partial
    sums of one leave the other's counters alone."""
    runs = []
    for k, (lens, nqs, Hq, H, D) in enumerate((([5000, 3000], [1, 1], 8, 1, 128), ([2600], [9], 4, 1, 64), ([4100], [6], 8, 2, 128))):
        q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, Hq, H, D, 32, BF, 60 + k, dev)
        want = ref.attention(q, pages, ks, vs, table, lens, nqs, 0.1, 0)
        runs.append((q, pages, ks, vs, table, kv_len, cu, max(nqs), want, attn_bounds(*want, BF, lens)[0]))
    need = max(mosaic.kv_attention_workspace(r[0], mosaic.KVCache(*r[1:4]), r[7]).numel() for r in runs)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    for _ in range(3):
        for q, pages, ks, vs, table, kv_len, cu, most, want, bound in runs:
            o, _ = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, most, 0.1, 0, BF, ws=ws)
            within(o, want[0], bound)


def test_cache_past_32_bits(dev, mosaic):
    """Slots whose bytes lie past 2^32 of the cache, written, read back and attended to."""
    H, D, P = 8, 128, 64
    per_page = mosaic.lib().mq_kv_cache_bytes(1, P, H, D)
    pages = 2 ** 32 // per_page + 40
    cache = mosaic.KVCache(torch.empty((pages, H, P // 16, 18 * D), dtype=torch.uint8, device=dev))
    n = 150
    table = torch.tensor([[pages - 1, pages - 17, pages - 3]], dtype=torch.int32, device=dev)
    tok = torch.arange(n, device=dev)
    slots = table[0, tok // P].long() * P + tok % P
    gen = torch.Generator().manual_seed(5)
    k, v = (torch.randn(n, H, D, generator=gen).to(BF).to(dev) for _ in range(2))
    mosaic.mq_kv_append(k, v, slots, cache)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    mosaic.mq_kv_read(cache, slots, ko, vo)
    for x, got in ((k, ko), (v, vo)):
        assert torch.equal(got.cpu(), torch.from_numpy(oracle_rows(x, None)[2]).to(BF))
    q = torch.randn(1, 16, D, generator=gen).to(BF).to(dev)
    want = ref.attention(q, cache.pages, None, None, table, [n], [1], 0.09, 0)
    o, _ = run_attn(mosaic, q, cache.pages, None, None, table, torch.tensor([n], dtype=torch.int32, device=dev), None, 1, 0.09, 0, BF, False)
    within(o, want[0], attn_bounds(*want, BF, [n])[0])


def test_page_past_31_bits(dev, mosaic):
    """A page so large that its heads, and records inside a head, lie further apart than 2^31
    bytes: written, read back and attended to at both ends of both heads."""
    H, D, P, n = 2, 128, 2 ** 24, 90
    cache = mosaic.KVCache(torch.empty((1, H, P // 16, 18 * D), dtype=torch.uint8, device=dev))
    gen = torch.Generator().manual_seed(6)
    for first in (0, P - n):
        slots = first + torch.arange(n, device=dev)
        k, v = (torch.randn(n, H, D, generator=gen).to(BF).to(dev) for _ in range(2))
        k2, v2 = (torch.randn(n, H, D, generator=gen).to(BF).to(dev) for _ in range(2))
        mosaic.mq_kv_append(k, v, slots, cache)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        mosaic.mq_kv_read(cache, slots, ko, vo)
        for x, got in ((k, ko), (v, vo)):
            assert torch.equal(got.cpu(), torch.from_numpy(oracle_rows(x, None)[2]).to(BF)), first
        mosaic.mq_qkv_append(k2, k2, v2, torch.empty_like(k2), slots, cache)  # without norms and rotation
        mosaic.mq_kv_read(cache, slots, ko, vo)
        for x, got in ((k2, ko), (v2, vo)):
            assert torch.equal(got.cpu(), torch.from_numpy(oracle_rows(x, None)[2]).to(BF)), first
    # the page's last tokens alone, through a window
    q = torch.randn(1, 16, D, generator=gen).to(BF).to(dev)
    K, V = (torch.from_numpy(oracle_rows(x, None)[2]).to(dev).double() for x in (k2, v2))
    z = torch.einsum("hgd,nhd->hgn", q[0].double().view(H, -1, D), K) * 0.09
    p = torch.softmax(z, -1)
    want, mass = torch.einsum("hgn,nhd->hgd", p, V), torch.einsum("hgn,nhd->hgd", p, V.abs())
    smax = (0.09 * torch.einsum("hgd,nhd->hgn", q[0].double().abs().view(H, -1, D), K.abs())).amax(-1)
    lse, vmax = torch.logsumexp(z, -1), torch.full_like(smax, float(V.abs().max()))
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.tensor([P], dtype=torch.int32, device=dev)
    o, _ = run_attn(mosaic, q, cache.pages, None, None, table, lens, None, 1, 0.09, n, BF, False)
    flat = [x.reshape(1, 16, *x.shape[2:]) for x in (want, lse, mass, smax, vmax)]
    within(o, flat[0], attn_bounds(*flat, BF, [n])[0])


def test_attention_leaves_other_rows(dev, mosaic):
    lens, nqs = [50, 20], [2, 3]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs(lens, nqs, 4, 2, 64, 16, HF, 31, dev)
    q = torch.cat((q, q[:3]))
    o, lse = run_attn(mosaic, q, pages, ks, vs, table, kv_len, cu, 3, 0.2, 0, HF)
    assert (o[5:] == 77).all() and (lse[5:] == 77).all() and (o[:5] != 77).any()


def test_attention_graphs_and_streams(dev, mosaic):
    """A captured call replayed with other inputs and lengths, and calls on two streams."""
    H, D, P, B = 2, 128, 16, 3
    lens = [200, 31, 90]
    q, pages, ks, vs, table, kv_len, cu = attn_inputs([256] * B, [1] * B, 8, H, D, P, BF, 41, dev)
    cache = mosaic.KVCache(pages, ks, vs)
    kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    out, ws = torch.empty_like(q).contiguous(), mosaic.kv_attention_workspace(q, cache, 1)
    call = lambda w=ws, o=out: mosaic.mq_kv_attention(q, cache, table, kv_len, o, 0.09, ws=w)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in (lens, [1, 256, 128], [0, 0, 5]):
        kv_len.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(sum(now))).to(BF))
        graph.replay()
        want = ref.attention(q, pages, ks, vs, table, now, [1] * B, 0.09, 0)
        within(out, want[0], attn_bounds(*want, BF, [256])[0], str(now))
    kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    call()
    torch.cuda.synchronize()
    outs = [torch.empty_like(out) for _ in range(2)]
    wss = [mosaic.kv_attention_workspace(q, cache, 1) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            mosaic.mq_kv_attention(q, cache, table, kv_len, outs[i], 0.09, ws=wss[i], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


# ------------------------------------------------------------------- all of them together
@pytest.mark.parametrize("norm", [True, False])
def test_attention_layer(norm, dev, mosaic):
    """A prompt of 40 tokens (quantized activations), then decode steps of two sequences and a
    step of three drafted tokens, against the same steps done in 64 bits from the values that
    the layers, the cache and every rounding hold."""
    Hq, H, D, hidden, P = 4, 2, 64, 256, 16
    qkv, out = mosaic.Layer((Hq + 2 * H) * D, hidden, 6, dev), mosaic.Layer(hidden, Hq * D, 4, dev)
    for i, l in enumerate((qkv, out)):
        W = to_dev(synth.weight(l.N, l.K, 70 + i, 74, 0.06, 40, 2, 8.0), dev)
        l.prepare_path(W, to_dev(synth.act(128, l.K, 80 + i, 84, 4, 5.0), dev))
    cache = mosaic.KVCache.alloc(12, P, H, D, dev)
    freq = (1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).to(dev)
    gen = torch.Generator().manual_seed(3)
    w = [(1 + 0.1 * torch.randn(D, generator=gen)).to(BF).to(dev) if norm else None for _ in range(2)]
    layer = mosaic.AttentionLayer(qkv, out, Hq, cache, freq, w[0], w[1])
    table = torch.tensor([[3, 7, 1, 0], [5, 2, 9, 4]], dtype=torch.int32, device=dev)
    lens = [0, 0]

    def step(nqs):
        T = sum(nqs)
        X = torch.randn(T, hidden, generator=gen).to(BF).to(dev)
        pos = torch.cat([lens[b] + torch.arange(n) for b, n in enumerate(nqs)]).to(dev)
        seq = torch.repeat_interleave(torch.arange(2), torch.tensor(nqs)).to(dev)
        slots = table[seq, pos // P].long() * P + pos % P
        for b, n in enumerate(nqs):
            lens[b] += n
        cu = torch.tensor([0] + list(np.cumsum(nqs)), dtype=torch.int32, device=dev)
        kv_len = torch.tensor(lens, dtype=torch.int32, device=dev)
        y = layer.step(X, pos, slots, table, kv_len, cu, max(nqs)).clone()
        # the same from the parts: projection, rotation, the cache's own bytes, attention
        proj = (qkv.forward_16bit(X) if T <= 16 else qkv.forward(X)).clone().view(T, -1, D)
        qr, mag = ref.norm_rope(proj[:, :Hq], w[0], 1e-6, pos, freq, D, False)
        kr, _ = ref.norm_rope(proj[:, Hq:Hq + H], w[1], 1e-6, pos, freq, D, False)
        ko, vo = torch.empty(T, H, D, dtype=BF, device=dev), torch.empty(T, H, D, dtype=BF, device=dev)
        mosaic.mq_kv_read(cache, slots, ko, vo)
        for got, src in ((ko, kr), (vo, proj[:, Hq + H:].double())):
            # a 4-bit value is off by at most 1/4 of its size, or 1/12 of its group's largest
            g = src.abs().reshape(T, H, -1, 16).amax(-1, keepdim=True).expand(-1, -1, -1, 16).reshape(src.shape)
            within(got, src, 0.25 * src.abs() + g / 6 * 0.25 * 1.1 + g * 0.07)
        qb = torch.empty(T, Hq, D, dtype=BF, device=dev)
        mosaic.mq_qk_norm_rope(proj[:, :Hq], None, qb, None, pos, freq, w[0], None)
        within(qb, qr, rope_bound(qr, mag, BF))
        a = ref.attention(qb, cache.pages, None, None, table, lens, nqs, D ** -0.5, 0)
        o = torch.empty(T, Hq, D, dtype=BF, device=dev)
        mosaic.mq_kv_attention(qb, cache, table, kv_len, o, D ** -0.5, cu, max(nqs),
                               ws=mosaic.kv_attention_workspace(qb, cache, max(nqs)))
        within(o, a[0], attn_bounds(*a, BF, lens)[0], "attention")
        z = out.forward_16bit(o.view(T, -1)) if T <= 16 else out.forward(o.view(T, -1))
        assert torch.equal(z, y)

    for nqs in ([23, 17], [1, 1], [1, 1], [3, 1], [0, 2], [9, 1]):
        step(nqs)


def prompt_layer(mosaic, dev, hidden=256, Hq=4, H=2, D=64, P=16, n=64):
    """A layer with a cache of n tokens for each of two sequences, and a call for its prompts."""
    qkv, proj = mosaic.Layer((Hq + 2 * H) * D, hidden, 6, dev), mosaic.Layer(hidden, Hq * D, 4, dev)
    for i, l in enumerate((qkv, proj)):
        l.prepare_path(to_dev(synth.weight(l.N, l.K, 40 + i, 44, 0.06, 40, 2, 8.0), dev), to_dev(synth.act(128, l.K, 46 + i, 48, 4, 5.0), dev))
    freq = (1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).to(dev)
    layer = mosaic.AttentionLayer(qkv, proj, Hq, mosaic.KVCache.alloc(2 * n // P, P, H, D, dev), freq)
    table = torch.arange(2 * n // P, dtype=torch.int32, device=dev).view(2, -1)

    def prompt(X, b=0, **more):
        T = X.shape[0]
        pos = torch.arange(T, device=dev)
        slots = table[b, pos // P].long() * P + pos % P
        cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
        lens = torch.tensor([T], dtype=torch.int32, device=dev)
        t = table[b:b + 1].contiguous()
        return lambda X=X: layer.step(X, pos, slots, t, lens, cu, T, **more)

    return layer, prompt


def tokens(T, seed, dev, hidden=256):
    return torch.randn(T, hidden, generator=torch.Generator().manual_seed(seed)).to(BF).to(dev)


def test_attention_layer_prompts_have_results_of_their_own(dev, mosaic):
    """A step's result stays as it is when the layer takes other prompts of as many tokens, on
    other streams too, and prompts of many lengths leave nothing behind in the layers."""
    layer, prompt = prompt_layer(mosaic, dev)
    Xs = [tokens(40, i, dev) for i in range(4)]
    want = [prompt(X)().clone() for X in Xs]
    got = [prompt(X)() for X in Xs]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(layer._project(layer.qkv, Xs[0]), layer.qkv.forward(Xs[0]))  # the path's own result
    kept = len(layer.qkv._act), len(layer.out._act)
    for T in range(17, 64):
        prompt(tokens(T, T, dev))()
    assert (len(layer.qkv._act), len(layer.out._act)) == kept
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [prompt(X, b, stream=s) for b, (X, s) in enumerate(zip(Xs, streams))]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [c() for c in calls]
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_attention_layer_strided_tokens(dev, mosaic):
    """Tokens that are rows of a wider tensor give what their copies give, few and many of them."""
    layer, prompt = prompt_layer(mosaic, dev)
    for T in (5, 16, 17, 40):
        wide = torch.randn(T, 256 + 72, generator=torch.Generator().manual_seed(T)).to(BF).to(dev)
        X = wide[:, 8:8 + 256]
        want = prompt(X.contiguous())()
        assert torch.equal(prompt(X)(), want), T
    for bad in (wide, wide[:, :128].contiguous(), X.float()):
        with pytest.raises(mosaic.MosaicError):
            prompt(bad)()


def test_layer_forward_fresh_and_its_workspace(dev, mosaic):
    """Numbers of tokens whose products need a workspace, in any order, eager and captured: the
    results of forward; one workspace a stream."""
    N, K = 2048, 4096
    layer = mosaic.Layer(N, K, 100, dev)
    gen = torch.Generator().manual_seed(3)
    layer.prepare_path((0.02 * torch.randn(N, K, generator=gen)).to(BF).to(dev), tokens(128, 5, dev, K))
    Ms = (48, 128, 17, 100, 48, 64, 128, 200, 64)
    assert sum(mosaic.lib().mq_gemm_workspace_bytes(M, N, K, 0) > 0 for M in Ms) > 5
    Xs = [tokens(M, M, dev, K) for M in Ms]
    want = [layer.forward(X).clone() for X in Xs]
    for _ in range(3):
        got = [layer.forward_fresh(X) for X in Xs]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert len(layer._ws) == 1
    flags = mosaic.MQ_GEMM_BASE_ONLY
    base = layer.forward(Xs[0], flags).clone()
    assert torch.equal(layer.forward_fresh(Xs[0], flags), base) and torch.equal(layer.forward_fresh(Xs[0]), want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [layer.forward_fresh(X) for X in Xs]
    assert len(layer._ws) == 1
    for _ in range(3):
        assert torch.equal(layer.forward_fresh(Xs[3]), want[3])
        graph.replay()
        assert torch.equal(layer.forward_fresh(Xs[3]), want[3])
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_layer_captured_call_keeps_its_buffers_to_itself(dev, mosaic):
    """A first call of some number of tokens inside a capture: eager calls of as many get buffers of
    their own, with a workspace that is zero before any replay."""
    N, K, M = 2048, 4096, 64
    layer = mosaic.Layer(N, K, 100, dev)
    gen = torch.Generator().manual_seed(4)
    layer.prepare_path((0.02 * torch.randn(N, K, generator=gen)).to(BF).to(dev), tokens(128, 5, dev, K))
    X, Z = tokens(M, 1, dev, K), tokens(M, 2, dev, K)
    layer.forward(tokens(M + 1, 1, dev, K))  # the library's first use, with another number of tokens
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(X)
        buf = layer.buffers(M, 128, slot=1)
    assert not any(key[0] == M for key in layer._act) and buf.ws_gemm == buf.act[2].data_ptr()
    eager = layer.forward(Z)
    assert eager.data_ptr() != out.data_ptr() and layer.forward(Z) is eager
    want, wantX = layer.forward_fresh(Z), layer.forward_fresh(X)
    for _ in range(3):
        graph.replay()
        assert torch.equal(eager, want) and torch.equal(out, wantX)
        assert torch.equal(layer.forward(Z), want) and torch.equal(out, wantX)


def test_attention_layer_captured_prompt_before_an_eager_one(dev, mosaic):
    """The first call of a number of tokens is captured; eager ones of as many do not meet the
    graph's memory, before a replay or after it."""
    layer, prompt = prompt_layer(mosaic, dev)
    X, Y = tokens(48, 1, dev), tokens(48, 2, dev)
    call, other = prompt(X, 0), prompt(Y, 1)
    prompt(tokens(20, 3, dev))()  # the library's first use, with other sizes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    eager = other()
    again = call().clone()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        assert torch.equal(other(), eager) and torch.equal(out, again)


def test_attention_layer_in_graphs(dev, mosaic):
    """Two captured steps of one layer and eager ones, in any order and at once: each has a
    workspace of its own, and a graph replayed first is not the one that was captured first."""
    Hq, H, D, hidden, P, n = 8, 1, 64, 128, 32, 3000
    qkv, proj = mosaic.Layer((Hq + 2 * H) * D, hidden, 3, dev), mosaic.Layer(hidden, Hq * D, 2, dev)
    for i, l in enumerate((qkv, proj)):
        l.prepare_path(to_dev(synth.weight(l.N, l.K, 90 + i, 94, 0.06, 40, 2, 8.0), dev), to_dev(synth.act(128, l.K, 96 + i, 98, 4, 5.0), dev))
    pages, _, _ = ref.random_cache(2 * (-(-n // P) + 1), P, H, D, 6, dev, False)
    freq = (1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).to(dev)
    layer = mosaic.AttentionLayer(qkv, proj, Hq, mosaic.KVCache(pages), freq)
    table = torch.arange(pages.shape[0], dtype=torch.int32, device=dev).view(2, -1)
    calls = []
    for b in range(2):  # the step of each sequence alone; the same token again at every call
        X = torch.randn(1, hidden, generator=torch.Generator().manual_seed(b)).to(BF).to(dev)
        pos = torch.tensor([n - 1], device=dev)
        slots = table[b, pos // P].long() * P + pos % P
        lens = torch.tensor([n], dtype=torch.int32, device=dev)
        calls.append(lambda X=X, pos=pos, slots=slots, t=table[b:b + 1].contiguous(), lens=lens: layer.step(X, pos, slots, t, lens))
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want[1])
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = calls[0]()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[0])
