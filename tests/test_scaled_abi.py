"""Host-side checks (no GPU) of scored routing and of the float8 block-scaled operators: every bad
argument is refused before anything is enqueued, and the plain forms used by the GPU tests agree
with torch's own e4m3 conversion."""
import ctypes

import numpy as np
import pytest

import scaled_ref as ref


@pytest.fixture(scope="module")
def moe():
    from expert_ffn_token_b200 import build
    build.build()
    from expert_ffn_token_b200 import moe as m
    return m


FAKE = 0x7f0000000000        # 256-aligned, never dereferenced: validation fails first


def test_route_scored_refuses(moe):
    L = moe.library()
    need = moe.route_workspace_size(4, 16, 2)

    def call(logits=FAKE, T=4, E=16, k=2, rule=None, ids=FAKE, ws=FAKE, nbytes=need, status=None,
             **r):
        rule = moe.RouteRule(**r) if rule is None else rule
        return L.moe_route_scored(logits, T, E, k, ctypes.addressof(rule), ids, FAKE, FAKE, FAKE,
                                  FAKE, None, status, ws, nbytes, None)

    before = moe.kernels_enqueued()
    bad = moe.ERR_INVALID_ARG
    assert call(logits=None) == bad and call(ids=None) == bad and call(ws=None) == bad
    assert call(T=0) == bad and call(E=0) == bad and call(k=0) == bad and call(k=17) == bad
    assert call(k=40, E=64) == bad                             # at most 32
    assert call(score=2) == bad and call(score=-1) == bad
    assert call(n_group=0) == bad and call(n_group=3) == bad and call(E=66, n_group=33) == bad
    assert call(n_group=4, topk_group=5) == bad and call(n_group=4, topk_group=0) == bad
    assert call(n_group=8, topk_group=1, k=3) == bad            # groups of two: no third expert
    assert call(group_top=0) == bad and call(group_top=3) == bad
    assert call(n_group=16, topk_group=16, group_top=2) == bad  # groups of one
    assert call(scale=float("nan")) == bad and call(scale=float("inf")) == bad
    assert call(E=8192) == moe.ERR_UNSUPPORTED
    assert call(logits=FAKE + 2) == moe.ERR_ALIGNMENT and call(ws=FAKE + 64) == moe.ERR_ALIGNMENT
    assert call(d_bias=FAKE + 1) == moe.ERR_ALIGNMENT and call(status=FAKE + 2) == moe.ERR_ALIGNMENT
    assert call(nbytes=need - 1) == moe.ERR_WORKSPACE
    assert L.moe_route_scored(FAKE, 4, 16, 2, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE,
                              need, None) == bad
    assert moe.kernels_enqueued() == before


def test_scaled_quantize_refuses(moe):
    L = moe.library()

    def call(x=FAKE, dt=0, T=4, K=100, ldx=100, q=FAKE, ldq=112, s=FAKE, lds=4, status=None):
        return L.moe_scaled_quantize(x, dt, T, K, ldx, q, ldq, s, lds, status, None)

    before = moe.kernels_enqueued()
    bad = moe.ERR_INVALID_ARG
    assert call(x=None) == bad and call(q=None) == bad and call(s=None) == bad
    assert call(dt=3) == bad and call(dt=-1) == bad and call(T=-1) == bad and call(K=0) == bad
    assert call(ldx=99) == bad and call(ldq=96) == bad and call(lds=3) == bad
    assert call(ldq=104) == moe.ERR_ALIGNMENT and call(q=FAKE + 8) == moe.ERR_ALIGNMENT
    assert call(x=FAKE + 2) == moe.ERR_ALIGNMENT and call(dt=1, x=FAKE + 1) == moe.ERR_ALIGNMENT
    assert call(s=FAKE + 2) == moe.ERR_ALIGNMENT and call(status=FAKE + 1) == moe.ERR_ALIGNMENT
    assert call(T=0) == moe.OK
    assert moe.kernels_enqueued() == before


def test_scaled_matmul_refuses(moe):
    L = moe.library()

    def call(a=FAKE, lda=112, s=FAKE, ldas=4, M=4, K=100, b=FAKE, ldb=112, bs=FAKE, N=10, out=FAKE,
             dt=0, ldo=10, status=None, ws=None, nbytes=0):
        return L.moe_scaled_matmul(a, lda, s, ldas, M, K, b, ldb, bs, N, out, dt, ldo, status, ws,
                                   nbytes, None)

    before = moe.kernels_enqueued()
    bad = moe.ERR_INVALID_ARG
    for name in ("a", "s", "b", "bs", "out"):
        assert call(**{name: None}) == bad, name
    assert call(M=-1) == bad and call(N=0) == bad and call(K=0) == bad and call(dt=5) == bad
    assert call(lda=96) == bad and call(ldb=96) == bad and call(ldas=3) == bad and call(ldo=9) == bad
    assert call(lda=104) == moe.ERR_ALIGNMENT and call(ldb=120) == moe.ERR_ALIGNMENT
    assert call(a=FAKE + 8) == moe.ERR_ALIGNMENT and call(b=FAKE + 4) == moe.ERR_ALIGNMENT
    assert call(out=FAKE + 2) == moe.ERR_ALIGNMENT and call(dt=2, out=FAKE + 1) == moe.ERR_ALIGNMENT
    assert call(s=FAKE + 2) == moe.ERR_ALIGNMENT and call(bs=FAKE + 2) == moe.ERR_ALIGNMENT
    assert call(ws=FAKE + 16) == moe.ERR_ALIGNMENT
    big = (1 << 31) - 16
    assert call(K=big, lda=big, ldb=big) == moe.ERR_UNSUPPORTED
    assert call(M=0) == moe.OK
    n = ctypes.c_size_t()
    assert L.moe_scaled_matmul_workspace_size(4, 0, 16, ctypes.byref(n)) == bad
    assert L.moe_scaled_matmul_workspace_size(4, 16, 16, None) == bad
    assert moe.kernels_enqueued() == before


def test_scaled_experts_refuses(moe):
    L = moe.library()

    def weights(hidden=64, ffn=32, n_experts=4, shared=0, **k):
        p = dict(d_gate=FAKE, d_up=FAKE, d_down=FAKE, d_gate_s=FAKE, d_up_s=FAKE, d_down_s=FAKE)
        p.update(k)
        return moe.ScaledWeights(hidden, ffn, n_experts, shared, *p.values())

    need = moe.scaled_experts_workspace_size(weights(), 4, 2)

    def call(w=None, x=FAKE, xdt=1, T=4, k=2, ids=FAKE, rw=FAKE, off=FAKE, inv=FAKE,
             gate=None, out=FAKE, odt=1, status=None, ws=FAKE, nbytes=need):
        w = weights() if w is None else w
        return L.moe_scaled_experts(ctypes.addressof(w), x, xdt, T, k, ids, rw, off, inv, gate, out, odt, status, ws, nbytes, None)

    before = moe.kernels_enqueued()
    bad = moe.ERR_INVALID_ARG
    for name in ("x", "ids", "rw", "off", "inv", "out", "ws"):
        assert call(**{name: None}) == bad, name
    for name in ("d_gate", "d_up", "d_down", "d_gate_s", "d_up_s", "d_down_s"):
        assert call(w=weights(**{name: None})) == bad, name
        odd = FAKE + (8 if not name.endswith("_s") else 2)
        assert call(w=weights(**{name: odd})) == moe.ERR_ALIGNMENT, name
    assert call(w=weights(hidden=72)) == bad and call(w=weights(ffn=40)) == bad
    assert call(w=weights(shared=2)) == bad and call(w=weights(n_experts=0)) == bad
    assert call(w=weights(n_experts=5000)) == moe.ERR_UNSUPPORTED
    assert call(w=weights(hidden=1 << 17)) == moe.ERR_UNSUPPORTED
    assert call(T=0) == bad and call(k=0) == bad and call(k=5) == bad and call(xdt=3) == bad
    assert call(odt=-1) == bad and call(gate=FAKE) == bad       # a gate without a shared expert
    assert call(T=1 << 24) == moe.ERR_UNSUPPORTED
    assert call(x=FAKE + 8) == moe.ERR_ALIGNMENT and call(out=FAKE + 4) == moe.ERR_ALIGNMENT
    assert call(ids=FAKE + 2) == moe.ERR_ALIGNMENT and call(ws=FAKE + 128) == moe.ERR_ALIGNMENT
    assert call(nbytes=need - 1) == moe.ERR_WORKSPACE
    n = ctypes.c_size_t()
    w = weights()
    size = L.moe_scaled_experts_workspace_size
    assert size(None, 4, 2, ctypes.byref(n)) == bad
    assert size(ctypes.addressof(w), 0, 2, ctypes.byref(n)) == bad
    assert size(ctypes.addressof(w), 4, 5, ctypes.byref(n)) == bad
    assert size(ctypes.addressof(w), 4, 2, None) == bad
    assert moe.kernels_enqueued() == before


def test_experts_workspace_covers_every_smaller_batch(moe):
    for shared in (0, 1):
        w = moe.ScaledWeights(64, 32, 40, shared, *[FAKE] * 6)
        sizes = [moe.scaled_experts_workspace_size(w, t, 6) for t in range(1, 70)]
        assert sizes == sorted(sizes)


def test_binding_constants_match_the_header(moe):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "moe.h")) as f:
        found = dict(re.findall(r"\bMOE_((?:DT|SCORE)_[A-Z0-9]+)\s*=\s*(\d+)", f.read()))
    assert len(found) == 5
    for name, val in found.items():
        assert getattr(moe, name) == int(val), name


def test_layer_refuses_tensors_of_another_form(moe):
    import torch
    with pytest.raises(ValueError):        # not on a CUDA device
        moe._contiguous(torch.zeros(2, 2), "x", (2, 2), torch.float32, 0)
    with pytest.raises(moe.MoeError):
        moe.dtype_of(torch.zeros(1, dtype=torch.float64))


def test_plain_e4m3_agrees_with_torch():
    import torch
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4000) * 100, ref.E4M3[:127], ref._MID, [0.0, 2.0 ** -10]])
    v = np.clip(np.concatenate([v, -v]), -448, 448).astype(np.float32)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn)
    assert np.array_equal(t.float().numpy().astype(np.float64), ref.E4M3[ref.encode(v.astype(np.float64))])


def test_quantize_refuses_sizes_whose_block_counts_pass_32_bits(moe):
    L = moe.library()
    big = (1 << 31) - 1
    up = 1 << 31
    assert L.moe_scaled_quantize(FAKE, 0, 1, big, big, FAKE, up, FAKE, 1, None, None) == \
        moe.ERR_UNSUPPORTED
    assert L.moe_scaled_quantize(FAKE, 0, big, 1, 1, FAKE, 16, FAKE, big, None, None) == \
        moe.ERR_UNSUPPORTED


def test_route_scored_refuses_tokens_whose_chunk_count_passes_32_bits(moe):
    L = moe.library()
    rule = moe.RouteRule()
    call = lambda T: L.moe_route_scored(FAKE, T, 1, 1, ctypes.addressof(rule), FAKE, FAKE,  # noqa: E731
                                        FAKE, FAKE, FAKE, None, None, FAKE, 1 << 60, None)
    assert call((1 << 31) - 1) == moe.ERR_UNSUPPORTED
    assert call((1 << 30) + 1) == moe.ERR_UNSUPPORTED


def test_wait_limit_is_settable_and_not_zero(moe):
    with pytest.raises(moe.MoeError) as e:
        moe.scaled_set_wait_limit(0)
    assert e.value.code == moe.ERR_INVALID_ARG
    moe.scaled_set_wait_limit(1)
    moe.scaled_set_wait_limit(2_000_000_000)       # the default


def test_tensor_core_products_wait_on_bounded_barriers_only():
    """A warp that gives up leaves its loop, so no other may wait for it at a hardware barrier, which
    has no limit.  The kernel's two __syncthreads are reached by every thread."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "expert_ffn_token_b200", "csrc", "k_scaled_tc.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"named_barrier|bar\.sync|barrier\.sync|barrier\.cta", code)
    body = code[code.index("k_scaled_tc(const TcArgs"):]
    assert len(re.findall(r"__syncthreads\(\)", code)) == 2 == body.count("__syncthreads()")


class CudaTensor:
    """What the binding asks of a tensor on a CUDA device, without one."""

    is_cuda = True

    def __init__(self, shape, dtype, device=0, pointer=FAKE):
        self.shape, self.dtype, self.device, self.pointer = tuple(shape), dtype, device, pointer

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def numel(self):
        return int(np.prod(self.shape))

    def data_ptr(self):
        return self.pointer


def test_route_rule_keeps_its_bias(moe):
    """A rule made from a tensor holds it: later calls do not read memory that was given back."""
    import gc
    import weakref

    import torch
    bias = CudaTensor((64,), torch.float32, pointer=FAKE + 512)
    gone = weakref.ref(bias)
    rule = moe.RouteRule(d_bias=bias)
    del bias
    gc.collect()
    assert gone() is not None and rule.d_bias == FAKE + 512
    del rule
    gc.collect()
    assert gone() is None
    assert moe.RouteRule(d_bias=FAKE).d_bias == FAKE and moe.RouteRule().d_bias is None
    with pytest.raises(ValueError):
        moe.RouteRule(d_bias=torch.zeros(64))                       # not on a CUDA device
    with pytest.raises(ValueError):
        moe.RouteRule(d_bias=CudaTensor((64,), torch.bfloat16))


def test_layer_refuses_calls_on_another_device_than_its_own(moe, monkeypatch):
    """Weights and workspace of a layer are on its device: tensors on another one, current or not, are
    refused before anything is launched."""
    import torch
    called = []
    monkeypatch.setattr(moe, "scaled_experts", lambda *a: called.append(a))
    monkeypatch.setattr(moe, "route_scored", lambda *a: called.append(a))
    monkeypatch.setattr(moe, "read_status", lambda *a: called.append(a))
    monkeypatch.setattr(moe, "_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))
    moe._fill_dtypes()
    layer = moe.ScaledExperts.__new__(moe.ScaledExperts)
    layer.device, layer.hidden, layer.n_experts, layer.k, layer.rule = 0, 32, 4, 2, moe.RouteRule()
    layer.weights, layer._status, layer._ws, layer.ws_bytes = None, FAKE, FAKE, 0
    layer.status_word = layer.route_ws = CudaTensor((1,), torch.int32)
    layer.route_bytes = 0

    def run(dev):
        i32, f32, on = torch.int32, torch.float32, dict(device=dev)
        layer.forward(CudaTensor((3, 32), f32, **on), CudaTensor((3, 2), i32, **on),
                      CudaTensor((3, 2), f32, **on), CudaTensor((5,), i32, **on), None,
                      CudaTensor((6,), i32, **on), out=CudaTensor((3, 32), f32, **on))

    current = 0
    run(0)
    layer.status()
    assert len(called) == 2
    with pytest.raises(ValueError):
        run(1)                                   # tensors elsewhere
    current = 1
    for dev in (0, 1):
        with pytest.raises(ValueError):
            run(dev)                             # the layer elsewhere
        with pytest.raises(ValueError):
            layer.route(CudaTensor((3, 4), torch.float32, device=dev))
    with pytest.raises(ValueError):
        layer.status()
    assert len(called) == 2


@pytest.mark.parametrize("dt", [0, 1, 2])
def test_empty_batches_need_no_addresses(moe, dt):
    """Zero rows are a call that does nothing, with the null addresses that empty tensors have; the
    other arguments are checked all the same."""
    L = moe.library()
    quantise = lambda K=100, ldq=112: L.moe_scaled_quantize(None, dt, 0, K, 100, None, ldq, None, 0,  # noqa: E731
                                                            None, None)
    product = lambda b=FAKE, N=10, ldb=112: L.moe_scaled_matmul(  # noqa: E731
        None, 112, None, 0, 0, 100, b, ldb, FAKE, N, None, dt, 10, None, None, 0, None)
    before = moe.kernels_enqueued()
    assert quantise() == moe.OK and product() == moe.OK
    assert quantise(K=0) == moe.ERR_INVALID_ARG and quantise(ldq=104) == moe.ERR_ALIGNMENT
    assert product(b=None) == moe.ERR_INVALID_ARG and product(N=0) == moe.ERR_INVALID_ARG
    assert product(ldb=120) == moe.ERR_ALIGNMENT
    assert moe.kernels_enqueued() == before
