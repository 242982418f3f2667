"""Refusals of the logits calls that need no GPU: with S = 0 nothing is launched and no
pointer is looked at, so the sizes alone decide. And pins of the float64 forms the GPU tests
compare with."""
import ctypes
import math

import pytest

import split_residual_vector_b200 as pkg
from split_residual_vector_b200 import build as lib_build

torch = pytest.importorskip("torch")
import logits_ref as ref  # noqa: E402

OK, EINVAL = 0, -1


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return pkg.library()


ROWS = dict(dtype=0, S=0, n=1, V=100, ss=100, sn=0)
BAD_ROWS = [dict(dtype=2), dict(dtype=-1), dict(S=-1), dict(n=-1), dict(n=65537), dict(V=0),
            dict(V=-5), dict(V=(3 << 17) + 1), dict(ss=-1), dict(sn=-1), dict(S=1 << 41),
            dict(sn=1 << 60)]


def rows(over):
    r = {**ROWS, **over}
    return [None, r["dtype"], r["S"], r["n"], r["V"], r["ss"], r["sn"]]


def logprob(lib, scale=1.0, k=0, tokens=None, logprob=None, **over):
    return lib.mimi_rvq_token_logprob(*rows(over), tokens, 0, 0, -1, scale, k, logprob, None, None,
                                      None, None, None, None)


def logprob_grad(lib, scale=1.0, ds=100, dn=100, g=None, **over):
    return lib.mimi_rvq_token_logprob_grad(*rows(over), None, 0, 0, -1, scale, g, None, None, None,
                                           ds, dn, None, None, None, None, None)


def distill(lib, scale=1.0, k=4, tail=0, tdt=0, **over):
    return lib.mimi_rvq_distill_topk(*rows(over), None, None, tdt, k, tail, scale, None, None, None)


def distill_grad(lib, scale=1.0, k=4, tail=0, tdt=0, ds=100, dn=100, **over):
    return lib.mimi_rvq_distill_topk_grad(*rows(over), None, None, tdt, k, tail, scale, None, None,
                                          ds, dn, None, None, None)


CALLS = [logprob, logprob_grad, distill, distill_grad]


@pytest.mark.parametrize("call", CALLS)
def test_sizes_are_checked_before_anything_else(lib, call):
    assert call(lib) == OK
    assert call(lib, n=0) == OK
    assert call(lib, V=1, ss=1) == OK
    assert call(lib, V=3 << 17, ss=3 << 17) == OK
    for over in BAD_ROWS:
        assert call(lib, **over) == EINVAL, over
    for scale in (0.0, -1.0, 1e31, math.inf, math.nan):
        assert call(lib, scale=scale) == EINVAL


def test_lists_and_gradients_are_checked(lib):
    assert logprob(lib, k=128) == OK
    for k in (-1, 129):
        assert logprob(lib, k=k) == EINVAL
    fake = ctypes.c_void_p(16)
    assert logprob(lib, logprob=fake) == EINVAL      # a logprob needs tokens
    assert logprob_grad(lib, g=fake) == EINVAL       # and so does its gradient
    for call in (distill, distill_grad):
        assert call(lib, k=128, tail=1, tdt=1) == OK
        for over in (dict(k=0), dict(k=129), dict(tail=2), dict(tail=-1), dict(tdt=2)):
            assert call(lib, **over) == EINVAL, over
    for call in (logprob_grad, distill_grad):
        assert call(lib, ds=-1) == EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_host_pointers_are_refused(lib, call):
    """S > 0 with no device memory: an argument error, not a crash."""
    assert call(lib, S=2) in (EINVAL, -3)


def test_python_refuses_host_tensors():
    x, tok = torch.zeros((2, 8)), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: pkg.token_logprobs(x, tok), lambda: pkg.token_logprobs_grad(x, tok),
              lambda: pkg.distill_topk(x, tok.view(2, 1), torch.zeros((2, 1))),
              lambda: pkg.distill_topk_grad(x, tok.view(2, 1), torch.zeros((2, 1)))):
        with pytest.raises(AssertionError):
            f()


# ------------------------------------------------------------------ pins of the float64 forms


def test_float64_forms_on_worked_examples():
    x = torch.tensor([[math.log(1.0), math.log(2.0), math.log(5.0), -math.inf]], dtype=torch.float64)
    r = ref.logprob(x, torch.tensor([1]))
    assert abs(r["lse"][0].item() - math.log(8)) < 1e-14
    assert abs(r["logprob"][0].item() - math.log(0.25)) < 1e-14
    h = -(0.125 * math.log(0.125) + 0.25 * math.log(0.25) + 0.625 * math.log(0.625))
    assert abs(r["entropy"][0].item() - h) < 1e-14
    ids, lp, _ = ref.top(x, 5)
    assert ids.tolist() == [[[2, 1, 0, -1, -1]]] and lp[0, 0, 3] == -math.inf
    # distillation: q = (3/4, 1/4) over tokens 2 and 0, p = (5/8, 1/8)
    t = torch.tensor([[math.log(3.0), 0.0]], dtype=torch.float64)
    ids = torch.tensor([[2, 0]])
    want = 0.75 * math.log(0.75 / 0.625) + 0.25 * math.log(0.25 / 0.125)
    loss, _, d, _ = ref.distill(x, ids, t)
    assert abs(loss.item() - want) < 1e-14
    assert torch.allclose(d.view(-1), torch.tensor([0.125 - 0.25, 0.25, 0.625 - 0.75, 0.0],
                                                   dtype=torch.float64), atol=1e-14)
    # with the tail: q = (0.5, 0.2), q_r = 0.3 against p_r = 0.25 (token 1)
    t = torch.tensor([[math.log(0.5), math.log(0.2)]], dtype=torch.float64)
    want = 0.5 * math.log(0.5 / 0.625) + 0.2 * math.log(0.2 / 0.125) + 0.3 * math.log(0.3 / 0.25)
    loss, _, d, _ = ref.distill(x, ids, t, tail=True)
    assert abs(loss.item() - want) < 1e-14
    assert torch.allclose(d.view(-1), torch.tensor([0.125 - 0.2, 0.25 - 0.3, 0.625 - 0.5, 0.0],
                                                   dtype=torch.float64), atol=1e-14)


@pytest.mark.parametrize("tail", [False, True])
def test_float64_gradients_are_autograd_s(tail):
    torch.manual_seed(0)
    x = torch.randn((3, 2, 9), dtype=torch.float64, requires_grad=True)
    tok = torch.randint(0, 9, (3, 2))
    a, b, z = torch.randn((3, 3, 2), dtype=torch.float64)
    c = 1.3
    lse = torch.logsumexp(c * x, -1)
    lp = (c * x - lse.unsqueeze(-1))
    f = (a * lp.gather(-1, tok.unsqueeze(-1)).squeeze(-1) + z * lse
         - b * (lp.exp() * lp).sum(-1)).sum()
    want, = torch.autograd.grad(f, x, retain_graph=True)
    assert torch.allclose(ref.logprob_grad(x.detach(), tok, a, b, z, c=c)[0], want, atol=1e-13)
    ids = torch.tensor([[[0, 3, 5], [1, 1, 2]], [[-1, 4, 8], [7, 6, 5]], [[0, 1, 2], [8, 8, 8]]])
    t = torch.log_softmax(torch.randn((3, 2, 5), dtype=torch.float64), -1)[..., :3] - 1.0
    there = ids >= 0
    tm = torch.where(there, t, -math.inf)
    at = ids.clamp_min(0)
    if tail:
        q = tm.exp()
        qr = 1 - q.sum(-1)
        inside = torch.zeros((3, 2, 9)).scatter_add_(-1, at, there.float()) > 0
        rest = torch.logsumexp(torch.where(inside, -math.inf, c * x), -1) - lse
        f = torch.where(there, q * (t - lp.gather(-1, at)), 0.0).sum(-1) + qr * (qr.log() - rest)
    else:
        lq = torch.log_softmax(tm, -1)
        f = torch.where(there, lq.exp() * (torch.where(there, lq, 0.0) - lp.gather(-1, at)),
                        0.0).sum(-1)
    want, = torch.autograd.grad((a * f).sum(), x)
    loss, _, d, _ = ref.distill(x.detach(), ids, t, a, tail, c)
    assert torch.allclose(loss, f.detach(), atol=1e-13)
    assert torch.allclose(d, want, atol=1e-13)
