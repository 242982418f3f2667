"""The calls on the streams' logits at the edges of what they allow: layouts that lie between one
another, extreme logits and scales, optional arguments, and many rows with long lists."""
import pytest

torch = pytest.importorskip("torch")
import logits_ref as ref  # noqa: E402
from logits_ref import near  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32 = torch.bfloat16, torch.float32


def pkg():
    import split_residual_vector_b200 as p
    return p


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, seed, spread=3.0):
    return torch.empty(shape, device="cuda").normal_(0, spread, generator=gen(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [6, 2048, 6001, 140001])
def test_tail_class_between_logits_of_opposite_sign(V, dtype):
    """Listed logits near float32's largest value and the others near its lowest: the tail's log
    probability is the scale times a difference that float32 does not hold."""
    p = pkg()
    x = normal((4, V), dtype, 1) * 1e30 - 3.0e38
    ids = torch.stack([torch.randperm(V, device="cuda", generator=gen(i))[:4] for i in range(4)])
    ids = ids.to(torch.int32)
    x.scatter_(1, ids.long(), 3.0e38)
    t = torch.tensor([[0.4, 0.2, 0.1, 0.05]] * 4, device="cuda").log()
    for c in (0.5, 0.001):
        loss, t_loss, d, t_d = ref.distill(x, ids, t, None, True, c)
        assert torch.isfinite(loss).all() and (loss > 1e34).all()
        near(p.distill_topk(x, ids, t, tail=True, scale=c), loss, t_loss, f"loss {c}")
        got, l2 = p.distill_topk_grad(x, ids, t, tail=True, scale=c, loss=True)
        near(l2, loss, t_loss, f"loss with gradient {c}")
        near(got, d, t_d, f"dlogits {c}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [5, 300, 2048, 9001, 140001])
def test_logits_over_the_whole_range_at_the_smallest_scale(V, dtype):
    """Differences of logits past float32's range: probability 0 at every scale that is taken."""
    p = pkg()
    x = (normal((4, V), F32, 2, 1.0e38).clamp(-3.3e38, 3.3e38)).to(dtype)
    x[:, 0], x[:, V - 1] = 3.3e38, -3.3e38
    x[2:] = normal((2, V), F32, 3, 1.0e30).to(dtype)  # ordinary exponents at this scale
    tok = torch.tensor([0, V - 1, 1, V // 2], device="cuda", dtype=torch.int32)
    c = torch.tensor(1e-30).item()
    want = ref.logprob(x, tok, c=c)
    r = p.token_logprobs(x, tok, scale=c, top_k=min(V, 9))
    for name, (v, tol) in want.items():
        near(getattr(r, name), v, tol, name)
    ids, lp, tol = ref.top(x, min(V, 9), c)
    assert torch.equal(r.top_ids.long(), ids[:, 0])
    near(r.top_logprob, lp, tol, "top_logprob")
    ids = torch.tensor([[0, V // 2, 2]] * 4, device="cuda", dtype=torch.int32)
    t = torch.tensor([[0.4, 0.2, 0.1]] * 4, device="cuda").log()
    g = torch.full((4,), 1e30, device="cuda")  # gradients that float32 holds
    for tail in (False, True):
        loss, t_loss, d, t_d = ref.distill(x, ids, t, g, tail, c)
        near(p.distill_topk(x, ids, t, tail=tail, scale=c), loss, t_loss, f"loss {tail}")
        near(p.distill_topk_grad(x, ids, t, g, tail=tail, scale=c), d, t_d, f"dlogits {tail}")


@pytest.mark.parametrize("c", [9.9e-31, 1e-37, 1e-44])
def test_smaller_scales_are_refused(c):
    p = pkg()
    x = normal((3, 50), F32, 4)
    tok = torch.zeros(3, device="cuda", dtype=torch.int32)
    g = torch.ones(3, device="cuda")
    ids, t = tok.view(3, 1), g.view(3, 1)
    for call in (lambda: p.token_logprobs(x, tok, scale=c),
                 lambda: p.token_logprobs_grad(x, tok, g, scale=c),
                 lambda: p.distill_topk(x, ids, t, scale=c),
                 lambda: p.distill_topk_grad(x, ids, t, g, scale=c)):
        with pytest.raises(p.MimiRVQError):
            call()


def interleaved(S, n, V, dtype):
    """(name, x, d): views [S, n, V] of one buffer that share no element."""
    def two(shape, pick):
        buf = normal(shape, dtype, 3)
        return pick(buf)

    yield "beside each other", *two((S, n, 2, V), lambda b: (b[:, :, 0], b[:, :, 1]))
    yield "and the other way", *two((S, n, 2, V), lambda b: (b[:, :, 1], b[:, :, 0]))
    yield "column ranges", *two((S, n, 2 * V + 7), lambda b: (b[..., 3:3 + V], b[..., V + 5:2 * V + 5]))
    yield "halves of the streams", *two((S, 2 * n, V), lambda b: (b[:, :n], b[:, n:]))
    yield "every other stream", *two((S, 2 * n, V), lambda b: (b[:, ::2], b[:, 1::2]))
    yield "every other step", *two((2 * S, n, V), lambda b: (b[1::2], b[::2]))
    yield "stream by stream", *two((n, S, 2, V), lambda b: (b[:, :, 0].transpose(0, 1),
                                                            b[:, :, 1].transpose(0, 1)))
    # steps that are no whole number of rows apart
    def padded(b):
        return (b.as_strided((S, n, V), (2 * n * V + 11, 2 * V, 1)),
                b.as_strided((S, n, V), (2 * n * V + 11, 2 * V, 1), V))
    yield "padded steps", *two((S * (2 * n * V + 11) + V,), padded)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,n,V", [(1, 1, 40), (1, 3, 100), (5, 1, 33), (6, 4, 2049), (3, 2, 9000)])
def test_gradients_between_the_logits_rows(S, n, V, dtype):
    p = pkg()
    tok = torch.randint(0, V, (S, n), device="cuda", generator=gen(4), dtype=torch.int32)
    g = torch.randn((S, n), device="cuda", generator=gen(5))
    ids = torch.randint(0, V, (S, n, 3), device="cuda", generator=gen(6), dtype=torch.int32)
    t = torch.full((S, n, 3), -1.5, device="cuda")
    for name, x, d in interleaved(S, n, V, dtype):
        kept = x.clone()
        assert p.token_logprobs_grad(x, tok, g, g, out=d) is d
        near(d, *ref.logprob_grad(kept, tok, g, g), name)
        assert torch.equal(x, kept), name
        p.distill_topk_grad(x, ids, t, g, tail=True, out=d)
        near(d, *ref.distill(kept, ids, t, g, True)[2:], name)
        assert torch.equal(x, kept), name


def test_gradients_that_share_elements_with_the_logits_are_refused():
    p = pkg()
    S, n, V = 4, 3, 50
    tok = torch.zeros((S, n), device="cuda", dtype=torch.int32)
    g = torch.ones((S, n), device="cuda")
    ids, t = tok.unsqueeze(-1), torch.zeros((S, n, 1), device="cuda")
    buf = torch.zeros(8 * S * n * V, device="cuda")
    view = lambda ss, sn, at: buf.as_strided((S, n, V), (ss, sn, 1), at)  # noqa: E731
    P, q = 2 * n * V, 2 * V
    for x, d in ((view(P, q, 0), view(P, q, V - 1)), (view(P, q, 0), view(P, q, V + 1)),
                 (view(P, q, V), view(P, q, 1)), (view(P, q, 0), view(P, q, 2 * V)),
                 (view(P, q, 0), view(P, q, P)), (view(P, q, 0), view(P + V, q, V)),
                 (view(P, q, V), view(P, V, 0)),
                 (view(P - V, q, 0), view(P - V, q, V)),   # a step's last row meets the next step
                 (view(P - V, q, V), view(P - V, q, 0))):
        with pytest.raises(p.MimiRVQError):
            p.token_logprobs_grad(x, tok, g, out=d)
        with pytest.raises(p.MimiRVQError):
            p.distill_topk_grad(x, ids, t, g, out=d)


def test_losses_that_are_not_wanted():
    p = pkg()
    x = normal((3, 50), F32, 7)
    ids = torch.zeros((3, 1), device="cuda", dtype=torch.int32)
    t = torch.zeros((3, 1), device="cuda")
    d = p.distill_topk_grad(x, ids, t, loss=False)
    assert torch.equal(d, p.distill_topk_grad(x, ids, t))


def test_arguments_past_the_calls_integers():
    """Sizes that a 32-bit argument would not hold are refused, not taken modulo 2^32."""
    p = pkg()
    x = normal((2, 50), F32, 8)
    tok = torch.full((2,), 5, device="cuda", dtype=torch.int32)
    for pad in ((1 << 32) + 5, -(1 << 32) + 5, 1 << 31):
        with pytest.raises(AssertionError):
            p.token_logprobs(x, tok, pad=pad)
        with pytest.raises(AssertionError):
            p.token_logprobs_grad(x, tok, torch.ones(2, device="cuda"), pad=pad)
    for pad in ((1 << 31) - 1, -(1 << 31)):
        assert p.token_logprobs(x, tok, pad=pad).logprob.all()
    wide = x[:1, :1].view(1, 1, 1).expand(1, (1 << 32) + 1, 1)[:, :, :1]
    with pytest.raises(AssertionError):
        p.token_logprobs(wide, out=p.TokenLogprobs(None, None, None, None, None))
    with pytest.raises(p.MimiRVQError):
        p.token_logprobs(x[:0], tok[:0], top_k=(1 << 32) + 1)


GRIDS = [(4000, 0, 12000, BF16, 8), (4000, 0, 5000, F32, 8), (2000, 8, 2048, BF16, 64),
         (2000, 8, 2048, BF16, 20), (2000, 8, 300, F32, 100), (3000, 0, 3000, F32, 33),
         (2000, 0, 20000, BF16, 128), (1500, 0, 32000, BF16, 64)]


@pytest.mark.parametrize("S,n,V,dtype,k", GRIDS)
def test_grids_of_many_rows_are_resident(S, n, V, dtype, k):
    """Rows are dealt out to the CTAs of the grid, so every CTA has to run from the start: the
    grid of a captured launch is compared with the CTAs the driver says fit."""
    driver = pytest.importorskip("cuda.bindings.driver")
    p = pkg()
    x = normal((S, max(n, 1), V), dtype, 9)
    x = x if n else x[:, 0]
    lead = x.shape[:-1]
    tok = torch.zeros(lead, device="cuda", dtype=torch.int32)
    ids = torch.randint(0, V, (*lead, k), device="cuda", generator=gen(10), dtype=torch.int32)
    t = torch.full(ids.shape, -6.0, device="cuda")
    g = torch.ones(lead, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def ok(result):
        assert result[0] == driver.CUresult.CUDA_SUCCESS, result[0]
        return result[1:]

    for name, call in (("values", lambda: p.token_logprobs(x, tok)),
                       ("alternatives", lambda: p.token_logprobs(x, tok, top_k=k)),
                       ("gradient", lambda: p.token_logprobs_grad(x, tok, g)),
                       ("loss", lambda: p.distill_topk(x, ids, t)),
                       ("loss's gradient", lambda: p.distill_topk_grad(x, ids, t, g))):
        call()
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(graph):
            call()
        raw = driver.CUgraph(graph.raw_cuda_graph())
        (count,) = ok(driver.cuGraphGetNodes(raw))[1:]
        nodes = ok(driver.cuGraphGetNodes(raw, count))[0]
        assert len(nodes) == 1, name
        (node,) = ok(driver.cuGraphKernelNodeGetParams(nodes[0]))
        func = node.func
        if int(func) == 0:
            (func,) = ok(driver.cuKernelGetFunction(node.kern))
        (fit,) = ok(driver.cuOccupancyMaxActiveBlocksPerMultiprocessor(func, node.blockDimX,
                                                                       node.sharedMemBytes))
        assert node.gridDimX <= fit * sms, f"{name}: {node.gridDimX} CTAs, {fit} fit an SM"
        del graph


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,n,V", [(10, 4, 2049), (1, 3, 50), (3, 1, 50), (4, 3, 1), (1, 1, 1),
                                   (0, 3, 50), (4, 0, 50)])
def test_new_gradients_are_laid_out_as_dense_logits(S, n, V, dtype):
    """Stream-major logits give stream-major gradients, so that each row's alignment is the
    logits' row's; all others, dense or not, contiguous ones."""
    p = pkg()
    dense = normal((n, S, V), dtype, 16).transpose(0, 1)
    layouts = [("streams", dense, dense.stride()), ("plain", dense.contiguous(), None),
               ("one row for all", normal((1, 1, V), dtype, 17).expand(S, n, V), None),
               ("padded", normal((n, S, V + 3), dtype, 18)[:, :, :V].transpose(0, 1), None)]
    for name, x, strides in layouts:
        tok = torch.zeros((S, n), device="cuda", dtype=torch.int32)
        g = torch.ones((S, n), device="cuda")
        d = p.token_logprobs_grad(x, tok, g)
        e = p.distill_topk_grad(x, tok.unsqueeze(-1), g.unsqueeze(-1), g)
        for out in (d, e):
            if strides is not None and S and n:
                assert out.stride() == strides, name
            else:
                assert out.is_contiguous() or 1 in (S, n, V), name
        if S and n:
            near(d, *ref.logprob_grad(x, tok, g), name)
            near(e, *ref.distill(x, tok.unsqueeze(-1), g.unsqueeze(-1), g)[2:], name)


@pytest.mark.parametrize("S,n,V,dtype", [(2500, 4, 300, BF16), (2500, 0, 2048, F32),
                                         (1900, 0, 6000, BF16), (1300, 0, 6000, F32),
                                         (1000, 0, 17001, BF16)])
def test_many_rows_with_long_lists(S, n, V, dtype):
    """Thousands of rows, so that every CTA walks several: ordinary rows between rows of few
    distinct values, whose alternatives overflow the list, and between lists with ids twice."""
    p = pkg()
    x = normal((S, max(n, 1), V), dtype, 11)
    few = torch.arange(S, device="cuda") % 3 == 1
    x[few] = torch.randint(-3, 3, x[few].shape, device="cuda", generator=gen(12)).to(dtype)
    x[torch.arange(S, device="cuda") % 7 == 2] = 1.5
    x = x if n else x[:, 0]
    lead = x.shape[:-1]
    for k in (24, 33, 64, 100, 128):
        r = p.token_logprobs(x, top_k=k)
        ids, lp, tol = ref.top(x, k)
        assert torch.equal(r.top_ids.reshape(ids.shape).long(), ids), k
        near(r.top_logprob, lp, tol, f"top {k}")
        del ids, lp, tol
    g = torch.randn(lead, device="cuda", generator=gen(13))
    for k in (20, 33, 64, 128):
        ids = torch.randint(0, V, (*lead, k), device="cuda", generator=gen(14), dtype=torch.int32)
        odd = torch.arange(S, device="cuda") % 2 == 1
        ids[odd, ..., 3::5] = ids[odd, ..., 1:2]
        ids[torch.arange(S, device="cuda") % 11 == 5] = -1
        t = torch.log_softmax(torch.randn(ids.shape, device="cuda", generator=gen(15)), -1) - 0.1
        for tail in (False, True):
            loss, t_loss, d, t_d = ref.distill(x, ids, t, g, tail)
            near(p.distill_topk(x, ids, t, tail=tail), loss, t_loss, f"loss {k}")
            got, l2 = p.distill_topk_grad(x, ids, t, g, tail=tail, loss=True)
            near(l2, loss, t_loss, f"loss with gradient {k}")
            near(got, d, t_d, f"dlogits {k}")
            del loss, d, t_d, got
