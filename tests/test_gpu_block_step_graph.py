"""A training step of a block's MLP half (norms with gate and stochastic depth, products, all gradients, clipping, weight
updates) captured once and replayed: the clipping plan is made outside the capture, over gradients that keep their memory."""
import pytest
import torch

from swin_window_attention_gb300 import capi

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from swin_window_attention_gb300 import build
    build.build()
    capi.load()


def _rand(seed, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std + mean).to(dtype).to(DEV)


@pytest.mark.parametrize("T,C", [(147, 96), (600, 192)])
def test_captured_and_replayed(T, C):
    f32 = torch.float32
    x, dy, dg = _rand(1, T, C), _rand(11, T, C, std=1e-2), _rand(12, T, C, std=1e-2)
    n1, n2 = [(_rand(s, C, std=0.2, mean=1.0, dtype=f32), _rand(s + 1, C, std=0.2, dtype=f32)) for s in (2, 4)]
    gate, keep = _rand(6, C, std=0.3, mean=0.7, dtype=f32), torch.tensor([1.25, 0.0, 1.25], device=DEV)
    w1, w2 = _rand(7, 4 * C, C, std=C ** -0.5), _rand(8, C, 4 * C, std=(4 * C) ** -0.5)
    b1, b2 = _rand(9, 4 * C, std=0.1, dtype=f32), _rand(10, C, std=0.1, dtype=f32)
    vec = lambda n=C: torch.empty(n, device=DEV)
    dw1, dw2, db1, db2 = torch.empty(4 * C, C, device=DEV), torch.empty(C, 4 * C, device=DEV), vec(4 * C), vec()
    ng1 = {"pre_weight": vec(), "pre_bias": vec()}
    ng2 = {"pre_weight": vec(), "pre_bias": vec(), "gate": vec()}
    grads = [dw1, dw2, db1, db2, *ng1.values(), *ng2.values()]
    clip = capi.GradClip(grads)  # once: it copies its list to the device and waits
    out = {"norm": torch.empty(1, device=DEV), "dx": torch.empty_like(x), "y": torch.empty_like(x),
           "u1": torch.empty(4 * C, C, dtype=torch.bfloat16, device=DEV), "u2": torch.empty(C, 4 * C, dtype=torch.bfloat16, device=DEV)}

    def step():
        _, h = capi.block_norm(x, pre=n1)
        pre = torch.empty(T, 4 * C, dtype=torch.bfloat16, device=DEV)
        a = capi.linear(h, w1, b1, act="gelu", pre=pre)
        f = capi.linear(a, w2, b2)
        y, _ = capi.block_norm(x, f, pre=n2, gate=gate, keep=keep, y=out["y"])
        dx, df, _ = capi.block_norm_bwd(y, f, dh=dg, dy=dy, pre=n2, gate=gate, keep=keep, grads=ng2, dx=out["dx"])
        capi.linear_bwd_weight(df, a, dw=dw2, db=db2)
        dpre = capi.linear_bwd_data(df, w2, pre=pre, act="gelu")
        capi.linear_bwd_weight(dpre, h, dw=dw1, db=db1)
        capi.block_norm_bwd(x, dh=capi.linear_bwd_data(dpre, w1), dy=dx, pre=n1, grads=ng1, dx=dx)
        clip(0.05, norm=out["norm"])
        capi.orthogonalize(dw1, out=out["u1"])
        capi.orthogonalize(dw2, out=out["u2"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    results = lambda: [t.clone() for t in (*grads, *out.values())]
    for seed, size in ((21, 1e-2), (31, 1e-6), (41, 3.0)):
        x.copy_(_rand(seed, T, C))
        dy.copy_(_rand(seed + 1, T, C, std=size))
        dg.copy_(_rand(seed + 2, T, C, std=size))
        for t in (*grads, *out.values()):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        got = results()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, results()))
        # clipped to 0.05 where they were longer (the last rounding, in fp32, of each)
        total = sum(float(t.double().square().sum()) for t in grads) ** 0.5
        norm = float(out["norm"])
        assert abs(total - min(norm, 0.05)) < 1e-4 * total and (norm > 0.05) == (size != 1e-6)
