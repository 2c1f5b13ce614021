"""The cache's operators together, as examples/decode_step.py runs them: the same logits
whichever way a sequence's tokens entered the cache (a prompt at once, token by token, a
verify step, after a fork with copy on write, after a compaction)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_step
    yield decode_step
    sys.path.remove(os.path.join(ROOT, "examples"))


def near(a, b, cache):
    """Both come from fp16 layers whose GEMMs and attention may sum in another order: a step
    (2^-10) at each of the 5 roundings of two layers, on the scale of the largest logit; with
    the int8 cache such a step can also move a code, 1 / 127 of its row's largest value, in a
    few of the values that a weight averages: four times that."""
    a, b = a.float(), b.float()
    steps = 2 * 5 * (4 if cache == "int8" else 1)
    return float((a - b).abs().max()) <= steps * 2.0 ** -10 * float(b.abs().max())


@pytest.mark.parametrize("cache", ["fp16", "int8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_one_sequence_many_ways(ex, cache, window, sinks):
    toks = [(53 * i + 7) % 1024 for i in range(50)]
    m = ex.Decoder(cache=cache)
    a = m.pool.add()
    whole = m.step([a], [toks], window, sinks)                       # the prompt at once
    b = m.pool.add()
    single = torch.cat([m.step([b], [[t]], window, sinks) for t in toks])
    assert near(single, whole, cache)
    c = m.pool.add()
    m.step([c], [toks[:37]], window, sinks)
    verify = m.step([c], [toks[37:43]], window, sinks)               # six tokens, then four rejected
    assert near(verify, whole[37:43], cache)
    m.pool.truncate(c, 39)
    f = m.pool.fork(c)                                               # shares a partly filled page
    two = m.step([c, f], [toks[39:41], [999]], window, sinks)
    assert near(two[:2], whole[39:41], cache)
    m.pool.free(a)
    m.pool.free(b)
    m.pool.free(f)
    before = {s: m.pool.table([s])[0].tolist() for s in (c,)}
    m.compact()
    assert m.pool.table([c])[0].tolist() != before[c]
    rest = m.step([c], [toks[41:]], window, sinks)
    assert near(rest, whole[41:], cache)


@pytest.mark.parametrize("cache", ["fp16", "int8"])
def test_example_runs(ex, cache, capsys):
    model, out, logits = ex.main(cache)
    assert len(out) == 4 and all(len(o) == 24 for o in out) and len({o[0] for o in out}) == 4
    assert torch.isfinite(logits.float()).all() and logits.shape == (2, model.vocab)
    assert "verify" in capsys.readouterr().out


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("first", [0, 1])
def test_decode_and_verify_graphs_in_turn(ex, own, first):
    """A decode step and a verify step, each captured into a graph of its own, with no workspace
    given or with one that only the smaller step has sized, then replayed in turn: the eager
    calls' bits.  The verify step's attention needs four times the workspace."""
    q, dev = ex.q, ex.DEV
    g = torch.Generator(device=dev).manual_seed(3)
    k, v = torch.randn(2, 400, 2, 16, 128, generator=g, device=dev).half()
    lens = torch.tensor([3000, 70, 1500], dtype=torch.int32, device=dev)
    table = torch.stack([torch.randperm(400, generator=g, device=dev)[:190].int() for _ in range(3)])
    ws = [q.Workspace(dev), q.Workspace(dev)] if own else [None, None]

    def step(new, vocab):
        cu = torch.arange(0, 3 * new + 1, new, dtype=torch.int32, device=dev)
        x = torch.randn(3 * new, 16, 128, generator=g, device=dev).half()
        y = torch.randn(3 * new, vocab, generator=g, device=dev).half()
        tok = torch.zeros(3 * new, dtype=torch.int32, device=dev)

        def run():
            return (q.attn_paged(x, k, v, table, lens, cu, max_new=new, ws=ws[0]),
                    *q.token_logprobs(y, tok, k=8, ws=ws[1]))
        return run
    steps = [step(1, 3000), step(6, 70000)]
    if own:
        steps[0]()
    torch.cuda.synchronize()
    graphs, outs = [None, None], [None, None]
    for i in (first, 1 - first):
        graphs[i] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[i]):
            outs[i] = steps[i]()
    junk = [torch.full((1 << 22,), 0x3f, dtype=torch.uint8, device=dev) for _ in range(8)]   # over what was given back
    want = [s() for s in steps]
    for i in (1 - first, first, 0, 1, 1, 0):
        for o in outs[i]:
            o.fill_(-1)
        graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs[i], want[i]):
            assert torch.equal(a, b)
        again = steps[i]()
        assert all(torch.equal(a, b) for a, b in zip(again, want[i]))
    assert q.device_error() == 0 and len(junk) == 8


def test_one_workspace_for_every_kind_of_call(ex):
    """Log probabilities leave their parts where attention keeps its counters, the GEMM and the
    prefill attention write there too: a Workspace keeps them apart."""
    q, dev = ex.q, ex.DEV
    g = torch.Generator(device=dev).manual_seed(4)
    shared = q.Workspace(dev)
    k, v = torch.randn(2, 300, 2, 16, 128, generator=g, device=dev).half()
    table = torch.randperm(300, generator=g, device=dev)[None, :250].int().contiguous()
    lens, cu = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([4000], [0, 3]))
    x = torch.randn(3, 16, 128, generator=g, device=dev).half()
    y = torch.randn(700, 3000, generator=g, device=dev).half()
    tok = torch.zeros(700, dtype=torch.int32, device=dev)
    w4, w8 = (ex._weights(5120, 1024, torch.Generator().manual_seed(bits), bits) for bits in (4, 8))
    z = torch.randn(20, 1024, generator=g, device=dev).half()
    p = torch.randn(256, 6, 256, generator=g, device=dev).half()
    calls = [lambda ws: q.attn_paged(x, k, v, table, lens, cu, max_new=3, ws=ws),
             lambda ws: q.token_logprobs(y, tok, k=64, ws=ws),
             lambda ws: q.qgemm_w4a16(z, w4, 5120, 1024, ws=ws),
             lambda ws: q.qgemm_lm_head_topk(q.MODE_W8A16, z, w8, 5120, 1024, 20, ws=ws),
             lambda ws: q.attn_int8qk_prefill(p, p[:, :2].contiguous(), p[:, 2:4].contiguous(), ws=ws)]
    want = [f(q.Workspace(dev)) for f in calls]
    for i in (0, 1, 0, 2, 0, 3, 0, 4, 0, 1, 2, 1, 3, 2, 4, 3, 1, 4, 2, 3):
        got = calls[i](shared)
        for a, b in zip(got if isinstance(got, tuple) else (got,), want[i] if isinstance(want[i], tuple) else (want[i],)):
            assert torch.equal(a, b), i
    torch.cuda.synchronize()
    assert q.device_error() == 0


def test_captures_have_numbers(ex):
    """0 outside a capture, one number in a capture, another in the next."""
    q, dev = ex.q, ex.DEV
    seen = []
    x = torch.zeros(8, device=dev)

    def number():
        return int(q.lib().qw_stream_capture_id(torch.cuda.current_stream().cuda_stream))
    for _ in range(2):
        assert number() == 0
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            x += 1
            seen.append(number())
            x += 1
            assert number() == seen[-1]
    assert number() == 0 and seen[0] != seen[1] and all(seen)
