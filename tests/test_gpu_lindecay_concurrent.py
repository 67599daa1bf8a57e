"""GPU tests of lindecay and blocknorm captured in graphs, and called from several streams and
threads at once: the bits of one call after the other."""
import threading

import pytest
import torch

from test_gpu_lindecay import DEV, draw, on_gpu, sml  # noqa: F401  (sml is a fixture)

pytestmark = pytest.mark.gpu

SHAPES = [(2, 500, 90, 1, 64, 64), (2, 300, 80, 2, 128, 64), (1, 2200, 4, 4, 64, 64), (1, 40, 2, 1, 32, 40)]


def attention(sml, shape, dtype=torch.bfloat16, seed=0):  # noqa: F811
    """A call with its gradients, of new results each time."""
    d = on_gpu(draw(*shape, dtype, seed=seed))

    def run():
        st, ds = torch.empty_like(d["state_in"]), torch.empty_like(d["state_in"])
        o = sml.lindecay_fwd(d["q"], d["k"], d["v"], d["log_a"], state_in=d["state_in"], state_out=st)
        g = sml.lindecay_bwd(d["q"], d["k"], d["v"], d["log_a"], d["dO"], state_in=d["state_in"],
                             dstate_out=d["dstate_out"], dstate_in=ds)
        return [o, st, *g, ds]

    return run


def norms(sml, rows=300, D=512, group=64):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(D)
    y, x, gate, dx, dh = (torch.randn((rows, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(5))
    w = [torch.randn(D, generator=g, device=DEV) for _ in range(3)]

    def run():
        xn, h = sml.blocknorm_fwd(y, w[0], x, gate, w[1], w[2], group=group)
        return [xn, h, *sml.blocknorm_bwd(dx, y, w[0], dh=dh, x_new=xn, gate=gate, scale=w[1], w_pre=w[2], group=group)]

    return run


def step(sml):  # noqa: F811
    d = on_gpu(draw(3, 1, 8, 2, 64, 64, torch.bfloat16))
    q, k, v = (d[n][:, 0].contiguous() for n in ("q", "k", "v"))
    st = torch.empty_like(d["state_in"])

    def run():
        st.copy_(d["state_in"])
        return [sml.lindecay_decode_step(q, k, v, d["log_a"], st), st]

    return run


CALLS = {**{f"attention {s}": lambda m, s=s: attention(m, s) for s in SHAPES},
         "attention f32": lambda m: attention(m, (1, 700, 4, 2, 64, 64), torch.float32),
         "norms": norms, "norms, groups value by value": lambda m: norms(m, 40, 480, 48), "step": step}


@pytest.mark.parametrize("name", list(CALLS))
def test_captured(sml, name):  # noqa: F811
    run = CALLS[name](sml)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sml.loglinear_check_status() == 0


def test_on_several_streams(sml):  # noqa: F811
    """Launches whose CTAs need all SMs at once, and others, side by side."""
    runs = [attention(sml, s, seed=i) for i, s in enumerate(SHAPES)] + [norms(sml)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(8):
        for i, (r, s) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(s):
                got.append((i, r()))
    torch.cuda.synchronize()
    assert sml.loglinear_check_status() == 0
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_from_several_threads(sml):  # noqa: F811
    runs = [attention(sml, s, seed=i) for i, s in enumerate(SHAPES)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    if not all(torch.equal(a, b) for a, b in zip(runs[i](), want[i])):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad and not any(t.is_alive() for t in threads)
    assert sml.loglinear_check_status() == 0
