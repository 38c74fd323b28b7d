"""Steps of one action block on several streams, with stream= and in graphs,
against the same steps run one after the other: the same bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DIM, HQ, HKV, D, F, C = 512, 8, 2, 128, 1024, 96


@pytest.fixture(scope="module")
def blk():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import action_block
    return action_block


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("fmt", [None, "int4"])
def test_steps_on_two_streams(blk, fmt):
    g = torch.Generator(device="cuda").manual_seed(5)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda")
    block = blk.random_block(DIM, HQ, HKV, D, F, fmt, seed=8)
    tok = blk.FeatureTokens(8, 1 + 0.1 * mk(C), 0.1 * mk(C), (mk(DIM, C) / C ** 0.5).bfloat16(), 0.1 * mk(DIM))
    feats = [mk(3000 + 500 * i, C).bfloat16() for i in range(2)]
    xs = [mk(4, 16, DIM).bfloat16() for _ in range(2)]
    want = []
    for f, x in zip(feats, xs):
        k, v = block.observe(tok(f))
        y = x
        for _ in range(4):
            y = block.step(y, k, v)
        want.append(y.clone())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(5):
        print(f"[action block, two streams] fmt={fmt} rep={rep}", flush=True)
        kv = [block.observe(tok(f, stream=s), stream=s) for f, s in zip(feats, streams)]
        ys = list(xs)
        for _ in range(4):
            for i, s in enumerate(streams):
                ys[i] = block.step(ys[i], *kv[i], stream=s)
        # other work on the current stream takes whatever memory is free to it
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(_bits(ys[i]), _bits(want[i])), (rep, i)
        del junk


def test_graph_replay_beside_an_eager_step(blk):
    g = torch.Generator(device="cuda").manual_seed(6)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    block = blk.random_block(DIM, HQ, HKV, D, F, "int4", seed=9)
    k, v = mk(3000, HKV, D), mk(3000, HKV, D)
    xs = [mk(4, 16, DIM) for _ in range(2)]
    want = [block.step(x, k, v).clone() for x in xs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(xs[0], k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for rep in range(4):
        print(f"[action block, graph beside eager] rep={rep}", flush=True)
        graph.replay()
        other = block.step(xs[1], k, v, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(_bits(y), _bits(want[0])) and torch.equal(_bits(other), _bits(want[1])), rep
        y.zero_()
        torch.cuda.synchronize()
