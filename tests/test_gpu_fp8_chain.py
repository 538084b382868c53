"""The 8-bit operators together, as a program uses them: a training step of a norm, the
router, the 8-bit expert layer and their backward; a serving step captured in a graph; calls
from several threads and on streams of their own."""
import threading

import numpy as np
import pytest

import oracle
import synth
from oracle import fp8
from test_gpu_fp8 import cd, dev, host, moe, norm_depth, q_tensor, scale_tensor

pytestmark = pytest.mark.gpu


class Layer:
    """One layer's tensors: norm weight, router, experts in 8 bits, and every buffer of a step."""

    def __init__(self, N, H, I, E, K, seed, kind="e8m0", residual=True):
        import torch
        m = moe()
        rng = np.random.default_rng(seed)
        self.N, self.H, self.I, self.E, self.K, self.kind = N, H, I, E, K, kind
        self.x = dev(rng.standard_normal((N, H)), "bf16")
        self.z = dev(2 * rng.standard_normal((N, H)), "bf16") if residual else None
        self.weight = dev(1 + 0.2 * rng.standard_normal(H), "bf16")
        self.wr = dev(rng.standard_normal((H, E)) * H ** -0.5, "fp32")
        up, down = rng.standard_normal((E, H, 2 * I)) * H ** -0.5, rng.standard_normal((E, I, H)) * I ** -0.5
        self.qu, self.su = q_tensor((E, 2 * I, H)), scale_tensor((E, cd(2 * I), cd(H)), kind)
        self.qd, self.sd = q_tensor((E, H, I)), scale_tensor((E, cd(H), cd(I)), kind)
        m.moe_quantize_weights(dev(up, "bf16"), self.qu, self.su)
        m.moe_quantize_weights(dev(down, "bf16"), self.qd, self.sd)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.r = torch.empty(N, H, **bf) if residual else self.x
        self.y, self.q, self.s = torch.empty(N, H, **bf), q_tensor((N, H)), scale_tensor((N, cd(H)), kind)
        self.rstd = torch.empty(N, device="cuda")
        self.idx = torch.empty(N, K, dtype=torch.int32, device="cuda")
        self.wt = torch.empty(N, K, device="cuda")
        self.meta = m.Metadata(N, K, E, N * K)
        self.out, self.h = torch.empty(N, H, **bf), torch.empty(N * K, 2 * I, **bf)
        self.dy, self.dx = torch.empty(N, H, **bf), torch.empty(N, H, **bf)
        self.dweight = torch.empty(H, **bf)
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(m.moe_expert_forward_fp8_workspace(self.meta, H, I), **u8)
        self.wsn = torch.empty(max(1, m.moe_rmsnorm_backward_workspace(N, H)), **u8)
        self.wsr = torch.empty(max(1, m.moe_route_workspace(N, K, E)), **u8)

    def forward(self, logits=None, stream=None):
        m = moe()
        m.moe_rmsnorm_forward(self.x, self.weight, 1e-5, residual=self.z, residual_out=None if self.z is None else self.r,
                              y=self.y, q=self.q, scale=self.s, rstd=self.rstd, stream=stream)
        if logits is None:
            logits = self.y.float() @ self.wr
        m.moe_route(logits, self.meta, renormalize=True, topk_idx=self.idx, topk_weights=self.wt, workspace=self.wsr,
                    stream=stream, want_aux=False)
        m.moe_expert_forward_fp8(self.meta, self.q, self.s, self.qu, self.su, self.qd, self.sd, self.out, h_save=self.h,
                                 workspace=self.ws, stream=stream)
        return logits

    def norm_backward(self, dresidual=None, stream=None):
        moe().moe_rmsnorm_backward(self.dy, self.r, self.weight, self.rstd, self.dx, self.dweight, dresidual=dresidual,
                                   workspace=self.wsn, stream=stream)

    def results(self):
        import torch
        b = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t
        return {k: b(getattr(self, k)).clone() for k in ("r", "y", "q", "s", "rstd", "idx", "wt", "out", "h", "dx", "dweight")}


def same(a, b):
    import torch
    return [k for k in a if not torch.equal(a[k], b[k])]


@pytest.mark.parametrize("kind", ["e8m0", "fp32"])
@pytest.mark.parametrize("N,H,I,E,K", [(24, 256, 128, 8, 2), (900, 528, 272, 4, 2)])
def test_training_step(N, H, I, E, K, kind):
    """Forward against its 64-bit form from the 8-bit operands on; the experts' backward on the
    bf16 values that the 8-bit operands stand for, against the formula and against differences
    of the 64-bit layer; then the norm's. Differences: central ones of a step t along a
    direction d err by t^2/6 of a third derivative: with t 2^-10 under 10^-4 of the slope."""
    import torch
    m = moe()
    c = Layer(N, H, I, E, K, seed=N, kind=kind)
    c.forward()
    ref = oracle.build_metadata(c.idx.cpu().numpy(), c.wt.cpu().numpy(), E)
    P = int(ref["P"])
    assert P == N * K
    # operands' values; bf16 holds each (4 bits and a power of two)
    vx, ox = host(c.q) * fp8.spread(host(c.s), H), fp8.spread(host(c.s), H)
    ou, od = fp8.spread2(host(c.su), 2 * I, H), fp8.spread2(host(c.sd), H, I)
    vu, vd = host(c.qu) * ou, host(c.qd) * od
    ro, bo, rh, eh = fp8.experts(vx, ox, vu, ou, vd, od, ref["expert_frequency_offset"], ref["x_gather_idx"],
                                 c.wt.cpu().numpy().reshape(-1)[ref["s_scatter_idx"]], N)
    assert np.all(np.abs(host(c.out) - ro) <= bo * (1 + 1e-2))
    assert np.all(np.abs(host(c.h) - rh) <= (eh + np.abs(rh) * fp8.HALF["bf16"]) * (1 + 1e-2))
    # the experts' backward
    rng = np.random.default_rng(1)
    dout = dev(rng.standard_normal((N, H)), "bf16")
    bu, bd = np.ascontiguousarray(vu.transpose(0, 2, 1)), np.ascontiguousarray(vd.transpose(0, 2, 1))
    bx, tu, td = dev(vx, "bf16"), dev(bu, "bf16"), dev(bd, "bf16")
    assert np.array_equal(host(bx), vx) and np.array_equal(host(tu), bu)
    dwu, dwd, dtw = torch.empty_like(tu), torch.empty_like(td), torch.empty(N, K, device="cuda")
    m.moe_expert_backward(c.meta, c.idx, bx, tu, td, c.h, dout, c.dy, dwu, dwd, dtw)
    f = oracle.forward(vx, bu, bd, ref)
    g = oracle.backward(vx, bu, bd, host(dout), ref, f)
    for name, got, want in (("dx", c.dy, g["dx"]), ("dw_up", dwu, g["dw_up"]), ("dw_down", dwd, g["dw_down"])):
        assert np.max(np.abs(host(got) - want)) <= 2e-2 * np.max(np.abs(want)), name
    loss = lambda v: float((oracle.forward(v, bu, bd, ref)["out"] * host(dout)).sum())
    d = g["dx"] / np.sqrt((g["dx"] ** 2).mean())
    slope = (loss(vx + 2.0 ** -10 * d) - loss(vx - 2.0 ** -10 * d)) * 2.0 ** 9
    # <dx, d> sums N H terms that are off by at most 2e-2 max|dx| each, of either sign: their
    # own size is max|d| sum|d| 2e-2 at the most
    assert abs((host(c.dy) * d).sum() - slope) <= 2e-2 * np.abs(g["dx"]).max() * np.abs(d).sum()
    # the norm's backward, with the residual stream's gradient
    c.norm_backward(dresidual=dout)
    r, w, dy = host(c.r), host(c.weight), host(c.dy)
    rx, rw, mx, mw = fp8.rmsnorm_backward(dy, r, w, host(c.rstd), host(dout))
    half = fp8.HALF["bf16"] * (1 + 1e-3)
    assert np.all(np.abs(host(c.dx) - rx) <= mx * (H / 256 + 80) * fp8.U32 + np.abs(rx) * half)
    assert np.all(np.abs(host(c.dweight) - rw) <= mw * (N / 64 + 80) * fp8.U32 + np.abs(rw) * half)
    lossn = lambda r, w: float((fp8.rmsnorm(r, w, 1e-5)[0] * dy).sum() + (r * host(dout)).sum())
    for which, got in (("r", host(c.dx)), ("w", host(c.dweight))):
        d = rng.standard_normal(got.shape)
        hi, lo = (lossn(r + t * d, w) if which == "r" else lossn(r, w + t * d) for t in (2.0 ** -10, -2.0 ** -10))
        # each term of <got, d> is off by half a step and the fp32 sums; rstd by norm_depth of
        # them; the difference itself by 1e-4
        size = (np.abs(d) * ((mx if which == "r" else mw) * (max(H, N) / 64 + 80 + 3 * norm_depth(H)) * fp8.U32
                             + np.abs(got) * half)).sum()
        slope = (hi - lo) * 2.0 ** 9
        assert abs((got * d).sum() - slope) <= size + 1e-4 * np.abs(got * d).sum()


@pytest.mark.parametrize("N,H,I,E,K", [(3, 256, 80, 8, 2), (1200, 528, 272, 3, 2)])
def test_graph_replays(N, H, I, E, K):
    """Forward and the norm's backward in one captured graph (the router's logits come in from
    outside), replayed over changing inputs with eager calls on the same layer, and other work,
    between the replays."""
    import torch
    c = Layer(N, H, I, E, K, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(0)
    inputs = [torch.randn(2, N, H, generator=gen, device="cuda").bfloat16() for _ in range(3)]

    logits = torch.empty(N, E, device="cuda")

    def step():
        c.forward(logits)
        c.norm_backward()

    def load(v):
        c.x.copy_(v[0])
        c.dy.copy_(v[1])
        logits.copy_(v[1][:, :E])

    want = []
    for v in inputs:
        load(v)
        step()
        torch.cuda.synchronize()
        want.append(c.results())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for graph in (g, g2):  # two graphs over the same workspaces, replayed in turn
        with torch.cuda.graph(graph, stream=s):
            step()
    other = torch.randn(512, 512, device="cuda")
    for rep in range(6):
        load(inputs[rep % 3])
        for t in (c.out, c.h, c.dx, c.dweight, c.y, c.rstd):
            t.fill_(float("nan"))
        c.ws.fill_(0xff)
        (other @ other).sum().item()
        (g if rep % 2 else g2).replay()
        torch.cuda.synchronize()
        assert not same(c.results(), want[rep % 3]), rep
        load(inputs[(rep + 1) % 3])
        step()  # eager, between replays
        torch.cuda.synchronize()
        assert not same(c.results(), want[(rep + 1) % 3])


def test_another_stream_than_the_current_one():
    """Every call with an explicit stream, behind work there that makes its inputs, while
    another stream is current."""
    import torch
    c = Layer(700, 528, 272, 3, 2, seed=2)
    logits = c.forward().clone()
    c.dy.normal_()
    c.norm_backward()
    torch.cuda.synchronize()
    want = c.results()
    x, dy = c.x.clone(), c.dy.clone()
    for t in (c.x, c.dy, c.out, c.h, c.y, c.dx, c.rstd):
        t.zero_()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):
            big = torch.tanh(big @ big)
        c.x.copy_(x)
        c.dy.copy_(dy)
    c.forward(logits, stream=s)
    c.norm_backward(stream=s)
    q, sc = q_tensor((700, 528)), scale_tensor((700, cd(528)), "e8m0")
    torch.cuda.current_stream().synchronize()
    moe().moe_quantize_rows(c.y, q, sc, stream=s)
    h, out = torch.empty_like(c.h), torch.empty_like(c.out)
    moe().moe_grouped_gemm_fp8(c.meta, c.q, c.s, c.qu, c.su, h, stream=s)
    moe().moe_expert_forward_fp8(c.meta, c.q, c.s, c.qu, c.su, c.qd, c.sd, out, stream=s)  # a workspace of its own
    s.synchronize()
    assert not same(c.results(), want)
    assert torch.equal(h, want["h"]) and torch.equal(out, want["out"])
    rq, rs = fp8.quantize_rows(host(c.y))
    assert np.array_equal(host(q), rq) and np.array_equal(host(sc), rs)


def test_threads_on_own_streams():
    import torch
    shapes = [(3, 512, 80, 16, 2), (900, 528, 272, 3, 2), (64, 256, 64, 4, 2), (2000, 256, 128, 4, 2)]
    serial = []
    for i, sh in enumerate(shapes):
        c = Layer(*sh, seed=i, kind="fp32" if i % 2 else "e8m0")
        c.dy.copy_(c.x)
        c.forward()
        c.norm_backward()
        torch.cuda.synchronize()
        serial.append((c.results()))
    layers = [Layer(*sh, seed=i, kind="fp32" if i % 2 else "e8m0") for i, sh in enumerate(shapes)]
    for c in layers:
        c.dy.copy_(c.x)
    torch.cuda.synchronize()
    streams, start, errors = [torch.cuda.Stream() for _ in layers], threading.Barrier(len(layers)), []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                start.wait(timeout=60)
                for _ in range(4):
                    layers[i].forward()
                    layers[i].norm_backward()
            streams[i].synchronize()
        except BaseException as ex:
            errors.append((i, ex))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(layers))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    for c, want in zip(layers, serial):
        assert not same(c.results(), want)


def test_timing_hook_names_the_kernels():
    """Events around the launches of one kernel at a time, for every kernel of these calls."""
    import torch
    m = moe()
    c = Layer(1500, 528, 272, 2, 2, seed=3)
    c.forward()
    torch.cuda.synchronize()
    for name, calls in (("rmsnorm", 1), ("up_swiglu_fp8", 1), ("down_fp8", 1), ("combine", 1), ("quant_rows", 0),
                        ("rmsnorm_bwd", 1), ("rmsnorm_dw", 1), ("grouped_fp8", 0), ("quant_weights", 0)):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
        m.moe_time_kernel(name, ev)
        c.forward()
        c.norm_backward()
        torch.cuda.synchronize()
        assert m.moe_time_kernel(name, None) == calls, name
