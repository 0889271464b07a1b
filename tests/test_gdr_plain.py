"""The 64-bit gated delta rule the GPU tests compare with: its gradients against
central differences of its forward, against automatic differentiation, and the
recurrence against the matrix form it stands for."""
import pytest

torch = pytest.importorskip("torch")

from tests import gdr_plain as plain  # noqa: E402


def _case(kind="random", carry=True):
    q, k, v, g, beta, h0 = plain.inputs(2, 5, 4, 2, 3, 6, seed=4, dtype=torch.float64, kind=kind, carry=carry)
    gen = torch.Generator().manual_seed(9)
    do = torch.randn(v.shape, generator=gen, dtype=torch.float64)
    dhT = torch.randn(2, 4, 3, 6, generator=gen, dtype=torch.float64)
    return [q, k, v, g, beta, h0.double()], do, dhT


@pytest.mark.parametrize("kind", ["random", "same_keys", "beta_edges", "zero_keys", "no_decay"])
def test_gradients_equal_automatic_differentiation(kind):
    args, do, dhT = _case(kind)
    leaves = [t.clone().requires_grad_() for t in args]
    o, hT = plain.forward(*leaves)
    want = torch.autograd.grad((o * do).sum() + (hT * dhT).sum(), leaves)
    got = plain.backward(*args[:5], do, h0=args[5], dhT=dhT)
    for name, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), want):
        torch.testing.assert_close(got[name], w, rtol=1e-11, atol=1e-12)


def test_gradients_equal_central_differences():
    args, do, dhT = _case()
    got = plain.backward(*args[:5], do, h0=args[5], dhT=dhT)
    step = 1e-6                     # error of a central difference: step^2 |f'''| + 2^-52 |f| / step, both near 1e-10 here
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        flat = args[i].reshape(-1)
        for j in range(0, flat.numel(), max(1, flat.numel() // 7)):
            f = []
            for s in (step, -step):
                moved = [t.clone() for t in args]
                moved[i].reshape(-1)[j] += s
                o, hT = plain.forward(*moved)
                f.append(float((o * do).sum() + (hT * dhT).sum()))
            assert abs((f[0] - f[1]) / (2 * step) - float(got[name].reshape(-1)[j])) < 1e-7, (name, j)


def test_recurrence_is_the_product_of_its_matrices():
    """S_t = a_t S_{t-1} (I - beta k k^T) + beta v k^T, with the matrices formed."""
    (q, k, v, g, beta, h0), _, _ = _case()
    o, hT = plain.forward(q, k, v, g, beta, h0)
    eye = torch.eye(6, dtype=torch.float64)
    for b in range(2):
        for h in range(4):
            S = h0[b, h]
            for t in range(5):
                kk = k[b, t, h // 2]
                S = g[b, t, h].exp() * S @ (eye - beta[b, t, h] * torch.outer(kk, kk)) + beta[b, t, h] * torch.outer(v[b, t, h], kk)
                torch.testing.assert_close(o[b, t, h], 6 ** -0.5 * S @ q[b, t, h // 2], rtol=1e-12, atol=1e-13)
            torch.testing.assert_close(hT[b, h], S, rtol=1e-12, atol=1e-13)


def test_norm_gradients_equal_central_differences():
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    for rms in (False, True):
        args = [rnd(3, 7), rnd(7), rnd(7), rnd(3, 7)]
        dy = rnd(3, 7)
        got = plain.norm_grads(*args, dy, rms=rms)
        for i, name in enumerate(("dx", "dweight", "dbias", "dz")):
            for j in range(0, args[i].numel(), 3):
                f = []
                for s in (1e-6, -1e-6):
                    moved = [t.clone() for t in args]
                    moved[i].reshape(-1)[j] += s
                    f.append(float((plain.norm(*moved, rms=rms)[0] * dy).sum()))
                assert abs((f[0] - f[1]) / 2e-6 - float(got[name].reshape(-1)[j])) < 1e-7, (name, j)
