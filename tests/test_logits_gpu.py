"""GPU parity of the operators on the streams' logits (token log probabilities, distillation
from a teacher's top list, their gradients) against plain float64 forms, through the C ABI."""
import math

import pytest

torch = pytest.importorskip("torch")
import logits_ref as ref  # noqa: E402
from logits_ref import near  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32 = torch.bfloat16, torch.float32
LOWEST = {BF16: torch.finfo(torch.bfloat16).min, F32: torch.finfo(torch.float32).min}


def pkg():
    import split_residual_vector_b200 as p
    return p


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(S, n, V, dtype, layout="plain", seed=0, spread=3.0):
    """Logits [S, n, V] ([S, V] for n = 0) in a memory layout."""
    g = gen(seed)
    m = max(n, 1)
    x = torch.empty((S, m, V), device="cuda").normal_(0, spread, generator=g).to(dtype)
    if layout == "streams":      # one stream after another
        x = x.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    elif layout == "offset":     # rows that start one element past an aligned address, gaps
        buf = torch.full((S * m * (V + 3) + 1,), math.nan, device="cuda", dtype=dtype)
        v = buf[1:].view(S, m, V + 3)[:, :, :V]
        v.copy_(x)
        x = v
    elif layout == "broadcast":  # every step reads the same row
        x = x[:1].expand(S, m, V)
    return x if n else x[:, 0]


def tokens_for(S, n, V, seed=1, pad=None):
    t = torch.randint(0, V, (S, max(n, 1)), device="cuda", generator=gen(seed), dtype=torch.int32)
    if pad is not None:
        t[4::5] = pad
    return t if n else t[:, 0]


def check_values(r, x, tokens, pad=-1, c=1.0, k=0):
    want = ref.logprob(x, tokens, pad, c)
    for name, (v, t) in want.items():
        near(getattr(r, name), v, t, name)
    if k:
        ids, lp, t = ref.top(x, k, c)
        assert torch.equal(r.top_ids.reshape(ids.shape).long(), ids)
        near(r.top_logprob, lp, t, "top_logprob")


SHAPES = [(1, 0, 1), (3, 0, 2), (5, 1, 7), (2, 3, 8), (4, 0, 31), (3, 2, 64), (2, 0, 255),
          (3, 5, 257), (9, 0, 1000), (130, 3, 2047), (37, 8, 2048), (11, 1, 2049), (5, 0, 4097),
          (3, 0, 8192), (1, 0, 10007), (2, 0, 16385), (1, 0, 32000), (300, 0, 32000),
          (7, 0, 32001), (2, 0, 65537), (1, 0, 131072), (3, 0, 262147), (2, 0, 3 << 17)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,n,V", SHAPES)
def test_logprob_values_and_alternatives(S, n, V, dtype):
    x = make(S, n, V, dtype, seed=V)
    tok = tokens_for(S, n, V, pad=V)
    for k, c in ((0, 1.0), (min(20, V + 2), 1.25)):
        r = pkg().token_logprobs(x, tok, pad=V, scale=c, top_k=k)
        check_values(r, x, tok, V, c, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["plain", "streams", "offset", "broadcast"])
@pytest.mark.parametrize("S,n,V", [(5, 3, 100), (6, 2, 2048), (3, 4, 2049), (4, 2, 9001)])
def test_logprob_layouts(S, n, V, layout, dtype):
    x = make(S, n, V, dtype, layout, seed=3)
    tok = tokens_for(S, n, V)
    check_values(pkg().token_logprobs(x, tok, top_k=5), x, tok, k=5)
    g = torch.randn((S, n), device="cuda", generator=gen(4))
    d = pkg().token_logprobs_grad(x, tok, g, g * 0.1, g * 0.2)
    near(d, *ref.logprob_grad(x, tok, g, g * 0.1, g * 0.2), "dlogits")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("k", [1, 2, 8, 31, 32, 33, 64, 65, 127, 128])
@pytest.mark.parametrize("S,V", [(4, 40), (5, 2048), (2, 5000), (3, 32001), (1, 150000)])
def test_top_alternatives_with_ties(S, V, k, dtype):
    """Few distinct logits, so that ties cross the list's end and every thread's share; rows of
    one value; -0 and +0 are the same."""
    g = gen(k)
    x = torch.randint(-40, 40, (S, V), device="cuda", generator=g).to(dtype)
    x[0] = 1.5
    if S > 1:
        x[1] = torch.where(torch.rand(V, device="cuda", generator=g) < 0.5, -0.0, 0.0).to(dtype)
    if S > 2:
        x[2] = torch.randint(0, 3, (V,), device="cuda", generator=g).to(dtype)
    if S > 3:  # ordinary values, few of them allowed
        x[3] = torch.where(torch.rand(V, device="cuda", generator=g) < 20.0 / V, x[3], -math.inf)
    r = pkg().token_logprobs(x, top_k=k)
    ids, lp, t = ref.top(x, k)
    assert torch.equal(r.top_ids.long(), ids[:, 0])
    near(r.top_logprob, lp, t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [130, 311, 600, 811, 2048, 2051, 4100, 32001])
def test_top_alternatives_of_ordinary_rows(V, dtype):
    """Every way the list's bound is found: from 32, 128 and 256 maxima, too few of them, and
    (sorted rows: one thread has all the largest) far too many logits above it."""
    x = make(6, 0, V, dtype, seed=V)
    x[1] = torch.sort(x[1].float(), descending=True).values.to(dtype)
    x[2] = torch.sort(x[2].float()).values.to(dtype)
    for k in (24, 25, 64, 65, 100, 128):
        r = pkg().token_logprobs(x, top_k=k)
        ids, lp, t = ref.top(x, k)
        assert torch.equal(r.top_ids.long(), ids[:, 0]), k
        near(r.top_logprob, lp, t, f"k {k}")


@pytest.mark.parametrize("S,n,V,dtype", [(9001, 3, 65, BF16), (3000, 7, 130, F32), (2500, 0, 4104, BF16),
                                         (2500, 0, 4104, F32), (1500, 0, 17001, BF16), (700, 0, 20001, F32),
                                         (130, 0, 70001, F32), (90, 0, 150001, BF16),
                                         (310, 0, 52001, BF16), (310, 0, 28001, F32),
                                         (160, 0, 60001, BF16)])
def test_many_rows(S, n, V, dtype):
    """More rows than are resident at once, so that every group walks several; among them rows
    without target, list or upstream gradient, and rows of NaN in their places."""
    p = pkg()
    x = make(S, n, V, dtype, seed=30)
    lead = x.shape[:-1]
    g = gen(31)
    off = torch.rand(lead, device="cuda", generator=g) < 0.3
    x[off & (torch.rand(lead, device="cuda", generator=g) < 0.2)] = math.nan
    tok = torch.where(off, V, tokens_for(S, n, V))
    r = p.token_logprobs(x, tok, pad=V, top_k=9)
    check_values(r, x, tok, V, k=9)
    check_values(p.token_logprobs(x, tok, pad=V), x, tok, V)
    a, b = torch.randn((2, *lead), device="cuda", generator=g)
    b[off] = 0
    b[torch.rand(lead, device="cuda", generator=g) < 0.5] = 0
    near(p.token_logprobs_grad(x, tok, a, b, pad=V), *ref.logprob_grad(x, tok, a, b, None, V))
    d, v = p.token_logprobs_grad(x, tok, a, pad=V, values=True)
    near(d, *ref.logprob_grad(x, tok, a, pad=V))
    check_values(v, x, tok, V)
    ids = torch.randint(0, V, (*lead, 21), device="cuda", generator=g, dtype=torch.int32)
    ids[off] = -1
    t = torch.log_softmax(torch.randn(ids.shape, device="cuda", generator=g), -1) - 0.2
    a[torch.rand(lead, device="cuda", generator=g) < 0.3] = 0
    for tail in (False, True):
        loss, t_loss, d, t_d = ref.distill(x, ids, t, a, tail)
        near(p.distill_topk(x, ids, t, tail=tail), loss, t_loss, "loss")
        near(p.distill_topk_grad(x, ids, t, a, tail=tail), d, t_d, "dlogits")
        got, l2 = p.distill_topk_grad(x, ids, t, a, tail=tail, loss=True)
        near(l2, loss, t_loss, "loss with gradient")
        near(got, d, t_d, "dlogits with loss")


def special_rows(V, dtype):
    """Rows on which a softmax can go wrong; NaN only in the rows from 7 on."""
    x = make(12, 0, V, dtype, seed=5)
    x[0] = -math.inf                 # nothing allowed
    x[1] = -math.inf
    x[1, V - 1] = 2.0                # one token allowed
    x[2] = LOWEST[dtype]             # masked by the type's lowest value: uniform
    x[3, ::2] = LOWEST[dtype]
    x[3, 1] = 5.0
    x[4, 1:] = -math.inf
    x[4, 0] = LOWEST[dtype]          # one allowed token, of the lowest value
    x[5, 0] = 3.0e38                 # a difference that overflows
    x[5, 1] = -3.0e38
    x[6] = 1.0e30
    x[7, V // 2] = math.nan
    x[8, 0] = math.inf
    x[9] = -math.inf
    x[9, 1] = math.nan
    x[10] = math.nan
    x[11, V - 1] = math.inf
    x[11, 0] = math.inf
    return x


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [5, 300, 2048, 7001, 40000, 140001])
def test_special_rows(V, dtype):
    p = pkg()
    x = special_rows(V, dtype)
    S = x.shape[0]
    tok = torch.full((S,), 1, device="cuda", dtype=torch.int32)
    for c in (1.0, 2.0, 0.5):
        check_values(p.token_logprobs(x, tok, scale=c, top_k=3), x, tok, c=c, k=3)
        one = torch.ones(S, device="cuda")
        for a, b, z in ((one, None, None), (one, one, None), (None, one, one)):
            d = p.token_logprobs_grad(x, tok, a, b, z, scale=c)
            near(d, *ref.logprob_grad(x, tok, a, b, z, c=c), f"c {c}")
    # no target: logprob 0, and no upstream gradient: zeros, whatever the row holds
    tok[:] = V
    r = p.token_logprobs(x, tok, pad=V)
    assert not r.logprob.any()
    d = p.token_logprobs_grad(x, tok, one, pad=V, out=x)  # in place
    assert d.data_ptr() == x.data_ptr() and not d.any()


def test_tokens_out_of_range_are_counted():
    p = pkg()
    x = make(6, 2, 50, F32)
    tok = tokens_for(6, 2, 50)
    tok[0, 0], tok[1, 1], tok[2, 0], tok[3, 0], tok[4, 1] = -1, 50, 51, 1 << 30, -(1 << 31)
    n_bad = torch.zeros(1, dtype=torch.int64, device="cuda")
    r = p.token_logprobs(x, tok, pad=50, n_bad=n_bad)
    check_values(r, x, tok, pad=50)
    assert int(n_bad.item()) == 2
    g = torch.ones((6, 2), device="cuda")
    d = p.token_logprobs_grad(x, tok, g, pad=50, n_bad=n_bad)
    near(d, *ref.logprob_grad(x, tok, g, pad=50))
    assert int(n_bad.item()) == 4
    ids = torch.tensor([[[50, 2], [-1, 3]]] * 6, dtype=torch.int32, device="cuda")
    p.distill_topk(x, ids, torch.zeros((6, 2, 2), device="cuda"), n_bad=n_bad)
    assert int(n_bad.item()) == 10


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,n,V", SHAPES)
def test_logprob_gradient(S, n, V, dtype):
    p = pkg()
    x = make(S, n, V, dtype, seed=V + 1)
    tok = tokens_for(S, n, V, pad=V)
    lead = x.shape[:-1]
    a, b, z = (torch.randn(lead, device="cuda", generator=gen(i)) for i in range(3))
    b[::3] = 0
    d, v = p.token_logprobs_grad(x, tok, a, b, z, pad=V, scale=0.75, values=True)
    near(d, *ref.logprob_grad(x, tok, a, b, z, V, 0.75), "all three")
    check_values(v, x, tok, V, 0.75)
    d = p.token_logprobs_grad(x, tok, a, pad=V)
    near(d, *ref.logprob_grad(x, tok, a, pad=V), "logprob")
    d = p.token_logprobs_grad(x, g_entropy=b)
    near(d, *ref.logprob_grad(x, None, None, b), "entropy")
    y = x.clone()
    d2 = p.token_logprobs_grad(y, tok, a, pad=V, out=y)
    assert d2 is y and torch.equal(y, p.token_logprobs_grad(x, tok, a, pad=V)), "in place"


def teacher_for(x, k, tail, seed=7, dtype=F32):
    """A teacher near the student: its top k ids and values, as token_logprobs gives them."""
    t = x.float() + 0.7 * torch.randn(x.shape, device="cuda", generator=gen(seed))
    r = pkg().token_logprobs(t.contiguous(), top_k=k)
    values = r.top_logprob if tail else torch.where(r.top_ids >= 0, r.top_logprob + 3.0, 0.0)
    return r.top_ids, values.to(dtype)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,n,V", SHAPES)
def test_distillation(S, n, V, dtype, tail):
    p = pkg()
    x = make(S, n, V, dtype, seed=V + 2)
    g = torch.randn(x.shape[:-1], device="cuda", generator=gen(8))
    for k in (1, 20, 128):
        ids, values = teacher_for(x, k, tail)
        ids[3::4] = -1  # steps without a teacher
        loss, t_loss, d, t_d = ref.distill(x, ids, values, g, tail, 0.8)
        near(p.distill_topk(x, ids, values, tail=tail, scale=0.8), loss, t_loss, f"loss {k}")
        got, l2 = p.distill_topk_grad(x, ids, values, g, tail=tail, scale=0.8, loss=True)
        near(l2, loss, t_loss, f"loss with gradient {k}")
        near(got, d, t_d, f"dlogits {k}")
        y = x.clone()
        assert torch.equal(p.distill_topk_grad(y, ids, values, g, tail=tail, scale=0.8, out=y), got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["plain", "streams", "offset", "broadcast"])
@pytest.mark.parametrize("S,n,V", [(5, 3, 100), (6, 2, 2048), (3, 4, 2049), (4, 2, 9001)])
def test_distillation_layouts(S, n, V, layout, dtype):
    p = pkg()
    x = make(S, n, V, dtype, layout, seed=9)
    for tail in (False, True):
        ids, values = teacher_for(x, 7, tail, dtype=BF16)
        loss, t_loss, d, t_d = ref.distill(x, ids, values, None, tail)
        got, l2 = p.distill_topk_grad(x, ids, values, tail=tail, loss=True)
        near(l2, loss, t_loss)
        near(got, d, t_d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [6, 2048, 5003, 70001])
@pytest.mark.parametrize("tail", [False, True])
def test_distillation_lists_that_go_wrong(V, dtype, tail):
    """Ids twice in a list, empty places with NaN, entries of -inf, lists without an entry, a
    student that forbids a listed token or everything, a certain student with a rest far below,
    NaN teachers, masked steps over broken rows."""
    p = pkg()
    x = make(14, 0, V, dtype, seed=10)
    ids = torch.stack([torch.randperm(V, device="cuda", generator=gen(i))[:5] for i in range(14)])
    ids = ids.to(torch.int32)
    t = torch.log_softmax(torch.randn((14, 5), device="cuda", generator=gen(11)), -1) - 0.3
    ids[0, 3] = ids[0, 1]                    # twice
    ids[1] = ids[1, 0]                       # five times
    ids[2, 2], t[2, 2] = -1, math.nan        # an empty place
    ids[3] = -1                              # no list, over a NaN row
    x[3, 0] = math.nan
    t[4, 1] = -math.inf                      # an entry without weight
    t[5] = -math.inf                         # a list without weight
    x[6, ids[6, 2].long()] = -math.inf       # a listed token that the student forbids
    x[7] = -math.inf                         # a student without a distribution
    x[8] = -200.0
    x[8, ids[8].long()] = 200.0              # all certainty in the list
    t[9, 0] = math.nan                       # a broken entry
    x[10, V // 2] = math.nan                 # a broken student
    x[11] = -math.inf                        # nothing outside the list
    x[11, ids[11].long()] = 1.0
    t[12] = math.log(0.2) + 1e-3             # more than 1 in all
    x[13] = LOWEST[dtype]                    # uniform
    g = torch.ones(14, device="cuda")
    loss, t_loss, d, t_d = ref.distill(x, ids, t, g, tail)
    near(p.distill_topk(x, ids, t, tail=tail), loss, t_loss, "loss")
    near(p.distill_topk_grad(x, ids, t, g, tail=tail), d, t_d, "dlogits")
    # weight 0: zeros even in the rows of NaN, and the losses are still given
    y, l2 = p.distill_topk_grad(x, ids, t, torch.zeros(14, device="cuda"), tail=tail, loss=True)
    assert not y.any()
    near(l2, loss, t_loss, "loss of weight 0")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [6, 2048, 40000])
def test_broken_entries_break_their_row(V, tail):
    p = pkg()
    x = make(4, 0, V, F32, seed=61)
    ids = torch.tensor([[0, 1, -1]] * 4, device="cuda", dtype=torch.int32)
    t = torch.full((4, 3), -1.5, device="cuda")
    t[0, 1], t[2, 0], t[3, 2] = math.inf, math.nan, math.inf  # the last one's place is empty
    d, l2 = p.distill_topk_grad(x, ids, t, tail=tail, loss=True)
    for loss in (p.distill_topk(x, ids, t, tail=tail), l2):
        assert torch.isnan(loss).tolist() == [True, False, True, False]
    assert torch.isnan(d).all(-1).tolist() == [True, False, True, False]
    assert torch.isfinite(d[1::2]).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [6, 2048, 40000])
def test_distillation_onto_the_lowest_logit(V, dtype, tail):
    """A listed token masked by the type's lowest value: a finite loss while its log probability
    is one in float32, infinite past it; the gradient is that of probability 0 either way."""
    p = pkg()
    x = make(3, 0, V, dtype, seed=60)
    x[:, 1] = LOWEST[dtype]
    ids = torch.tensor([[0, 1]] * 3, device="cuda", dtype=torch.int32)
    t = torch.tensor([[0.5, 0.25]] * 3, device="cuda").log()
    for c in (1.0, 2.0):
        loss, t_loss, d, t_d = ref.distill(x, ids, t, tail=tail, c=c)
        got_d, got = p.distill_topk_grad(x, ids, t, tail=tail, scale=c, loss=True)
        near(got_d, d, t_d, "dlogits")
        for v in (got, p.distill_topk(x, ids, t, tail=tail, scale=c)):
            if c == 1.0:
                near(v, loss, t_loss, "loss")
            else:
                assert (v == math.inf).all()


def test_distillation_of_the_whole_vocabulary():
    """A list that holds every token: the tail class is left out, the student's own
    distribution gives a loss of rounding size and the gradient of the full KL."""
    p = pkg()
    x = make(4, 0, 100, F32, seed=12)
    r = p.token_logprobs(x, top_k=100)
    for tail in (False, True):
        loss, t_loss, d, t_d = ref.distill(x, r.top_ids, r.top_logprob, None, tail)
        got, l2 = p.distill_topk_grad(x, r.top_ids, r.top_logprob, tail=tail, loss=True)
        near(l2, loss, t_loss)
        near(got, d, t_d)
        assert l2.abs().max().item() < 1e-5


def test_gradients_against_differences():
    """Central differences of the float64 forward, step h: their error is h^2 / 6 times a third
    derivative (below 24 c^3 (1 + ln V)^2 for these functions), plus 1e-15 / h of cancellation."""
    p = pkg()
    V, h, c = 11, 1e-3, 1.25
    x = make(3, 0, V, F32, seed=13, spread=1.0)
    tok = tokens_for(3, 0, V)
    a, b, z = 0.7, -0.4, 0.3
    one = torch.ones(3, device="cuda")
    slack = h * h * 4 * c ** 3 * (1 + math.log(V)) ** 2 + 1e-11

    def moved(f):
        out = torch.zeros((3, V), dtype=torch.float64, device="cuda")
        for i in range(V):
            e = torch.zeros(V, dtype=torch.float64, device="cuda")
            e[i] = h
            out[:, i] = (f(x.double() + e) - f(x.double() - e)) / (2 * h)
        return out

    def values(y):
        w = ref.logprob(y, tok, -1, c)
        return sum(k * w[name][0][:, 0] for k, name in ((a, "logprob"), (b, "entropy"), (z, "lse")))

    got = p.token_logprobs_grad(x, tok, a * one, b * one, z * one, scale=c)
    tol = ref.logprob_grad(x, tok, a * one, b * one, z * one, c=c)[1][:, 0]
    near(got, moved(values), tol + slack)
    for tail in (False, True):
        ids, t = teacher_for(x, 4, tail)
        got = p.distill_topk_grad(x, ids, t, tail=tail, scale=c)
        tol = ref.distill(x, ids, t, None, tail, c)[3][:, 0]
        near(got, moved(lambda y: ref.distill(y, ids, t, None, tail, c)[0][:, 0]), tol + slack)


def test_rows_beside_the_gradient_stay():
    """A gradient written into a strided view leaves what lies between its rows."""
    p = pkg()
    for dtype in (BF16, F32):
        for V in (9, 2047, 40001):
            x = make(5, 2, V, dtype, seed=14)
            buf = torch.full((5, 2, V + 5), 7.0, device="cuda", dtype=dtype)
            out = buf[:, :, 2:2 + V]
            tok = tokens_for(5, 2, V)
            g = torch.ones((5, 2), device="cuda")
            p.token_logprobs_grad(x, tok, g, out=out)
            near(out, *ref.logprob_grad(x, tok, g))
            ids, t = teacher_for(x, 3, True)
            p.distill_topk_grad(x, ids, t, tail=True, out=out)
            near(out, *ref.distill(x, ids, t, None, True)[2:])
            assert (buf[:, :, :2] == 7.0).all() and (buf[:, :, 2 + V:] == 7.0).all()


def test_rows_past_two_to_the_31_elements():
    p = pkg()
    V, far = 2049, (1 << 31) + 12345
    buf = torch.zeros(far + V, dtype=BF16, device="cuda")
    x = buf.as_strided((2, V), (far, 1))
    x.copy_(make(2, 0, V, BF16, seed=15))
    tok = tokens_for(2, 0, V)
    check_values(p.token_logprobs(x, tok, top_k=4), x.clone(), tok, k=4)
    ids, t = teacher_for(x.clone(), 4, True)
    want = ref.distill(x.clone(), ids, t, None, True)
    near(p.distill_topk_grad(x, ids, t, tail=True, out=x), *want[2:])


def test_same_bits_every_time_and_on_other_streams():
    p = pkg()
    for S, n, V, dtype in ((64, 0, 32000, BF16), (500, 8, 2048, F32), (1, 0, 131072, BF16)):
        x = make(S, n, V, dtype, seed=16)
        tok = tokens_for(S, n, V)
        g = torch.randn(x.shape[:-1], device="cuda", generator=gen(17))
        ids, t = teacher_for(x, 33, True)

        def run(stream=None):
            r = p.token_logprobs(x, tok, top_k=17, stream=stream)
            d = p.token_logprobs_grad(x, tok, g, g, stream=stream)
            e, loss = p.distill_topk_grad(x, ids, t, g, tail=True, loss=True, stream=stream)
            return (*r, d, e, loss)

        first = run()
        streams = [torch.cuda.Stream() for _ in range(3)]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        others = [run(s) for s in streams for _ in range(2)]
        torch.cuda.synchronize()
        for o in others:
            assert all(torch.equal(u, v) for u, v in zip(first, o))


def test_captured_graphs():
    """Two graphs over the same tensors, replayed in turn and at once with new values."""
    p = pkg()
    S, V, k = 40, 32001, 16
    x = make(S, 0, V, BF16, seed=18)
    tok = tokens_for(S, 0, V)
    g = torch.ones(S, device="cuda")
    r = p.token_logprobs(x, tok, top_k=k)
    d = p.distill_topk_grad(x, r.top_ids, r.top_logprob, g, tail=True)  # warm-up
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = p.token_logprobs(x, tok, top_k=k)
            d, loss = p.distill_topk_grad(x, r.top_ids, r.top_logprob * 0.5, g, tail=True, loss=True)
            e = p.token_logprobs_grad(x, tok, g, g)
        graphs.append(graph)
        outs.append((*r, d, loss, e))
    side = torch.cuda.Stream()
    for seed in (19, 20):
        x.copy_(make(S, 0, V, BF16, seed=seed))
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        r = p.token_logprobs(x, tok, top_k=k)
        d, loss = p.distill_topk_grad(x, r.top_ids, r.top_logprob * 0.5, g, tail=True, loss=True)
        want = (*r, d, loss, p.token_logprobs_grad(x, tok, g, g))
        for out in outs:
            assert all(torch.equal(u, v) for u, v in zip(want, out))


def test_argument_errors():
    p = pkg()
    x = make(4, 2, 64, F32)
    tok = tokens_for(4, 2, 64)
    ids, t = teacher_for(x, 3, False)
    for bad in (0.0, -1.0, 1e31, math.inf, math.nan):
        with pytest.raises(p.MimiRVQError):
            p.token_logprobs(x, tok, scale=bad)
    with pytest.raises(p.MimiRVQError):
        p.token_logprobs(x, tok, top_k=129)
    with pytest.raises(AssertionError):
        p.token_logprobs(x.transpose(1, 2), tok)          # a row's logits are not contiguous
    with pytest.raises(TypeError):
        p.token_logprobs(x.half(), tok)
    with pytest.raises(AssertionError):
        p.token_logprobs(x, tok.long())
    with pytest.raises(AssertionError):
        p.token_logprobs(x, tok[:3])
    with pytest.raises(AssertionError):
        p.token_logprobs(x.cpu(), tok)
    with pytest.raises(AssertionError):
        p.token_logprobs(x, tok.cpu())
    g = torch.ones((4, 2), device="cuda")
    with pytest.raises(p.MimiRVQError):                   # no tokens for their gradient
        p.token_logprobs_grad(x, None, g)
    with pytest.raises(p.MimiRVQError):                   # rows of the gradient share memory
        p.token_logprobs_grad(x, tok, g, out=torch.zeros((1, 2, 64), device="cuda").expand(4, 2, 64))
    buf = torch.zeros(4 * 2 * 64 + 8, device="cuda")
    y = buf[:512].view(4, 2, 64)
    with pytest.raises(p.MimiRVQError):                   # overlaps the logits, shifted
        p.token_logprobs_grad(y, tok, g, out=buf[8:].view(4, 2, 64))
    with pytest.raises(p.MimiRVQError):
        p.distill_topk_grad(y, ids, t, g, out=buf[4:516].view(4, 2, 64))
    with pytest.raises(p.MimiRVQError):
        p.distill_topk(x, torch.zeros((4, 2, 129), dtype=torch.int32, device="cuda"),
                       torch.zeros((4, 2, 129), device="cuda"))
    with pytest.raises(AssertionError):
        p.distill_topk(x, ids, t[..., :2])
    # nothing to do is no error
    e = p.token_logprobs(x[:0], tok[:0], top_k=4)
    assert e.logprob.shape == (0, 2) and e.top_ids.shape == (0, 2, 4)
    assert p.distill_topk_grad(x[:, :0], ids[:, :0].contiguous(), t[:, :0].contiguous()).numel() == 0


def test_streams_to_teacher_to_student():
    """The operators as they are used together: packed streams are embedded, a head gives the
    logits, a teacher's alternatives are kept, and a student learns from them and from the
    tokens read in place; columns of packed, pads included."""
    import synth
    p = pkg()
    text, audio = synth.moshi_streams(120, seed=21)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    packed = p.delay_pack(dev(text), dev(audio), [0, 1, 1, 1, 1, 1, 1, 1])
    rows = synth.moshi_rows()
    d_model = 64
    tables = torch.randn((sum(rows), d_model), device="cuda", generator=gen(22)).to(BF16)
    h = p.embed_sum(tables, rows, packed[:-1].contiguous(), out_dtype=F32)
    S = h.shape[0]
    head = torch.randn((8, d_model, 2048), device="cuda", generator=gen(23)) / 8
    logits = torch.einsum("sd,ndv->nsv", h, head).to(BF16).permute(1, 0, 2)  # stream by stream
    tok = packed[1:, 1:9]
    teacher = p.token_logprobs(logits, tok, pad=p.AUDIO_PAD, top_k=20)
    check_values(teacher, logits, tok, p.AUDIO_PAD, k=20)
    assert (teacher.logprob[-1, 1:] != 0).all() and teacher.logprob[-1, 0] == 0  # a pad's place
    student = (logits.float() + torch.randn((S, 8, 2048), device="cuda", generator=gen(24))).to(BF16)
    mask = (tok != p.AUDIO_PAD).float() / tok.numel()
    d, loss = p.distill_topk_grad(student, teacher.top_ids, teacher.top_logprob, mask, tail=True,
                                  loss=True)
    want = ref.distill(student, teacher.top_ids, teacher.top_logprob, mask, True)
    near(loss, *want[:2])
    near(d, *want[2:])
    e = p.token_logprobs_grad(student, tok, mask, pad=p.AUDIO_PAD)
    near(e, *ref.logprob_grad(student, tok, mask, pad=p.AUDIO_PAD))
    # a step along both gradients lowers the distillation loss of the whole batch
    total = float((loss * mask).sum())
    moved = (student.float() - 20.0 * d.float() / d.float().norm()).to(BF16)
    assert float((p.distill_topk(moved, teacher.top_ids, teacher.top_logprob, tail=True)
                  * mask).sum()) < total
