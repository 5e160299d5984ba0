"""fdllm_sample on the GPU against a row-by-row float64 sampler."""
import numpy as np
import pytest
import torch

from kv_cache_decode_dualcache_b200 import build, fdllm
from tests import kv8_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    build.build()


def _run(x, u, mask_id=-1, **filters):
    dev = {n: None if v is None else torch.as_tensor(
        v, dtype=torch.int32 if n == "top_k" else torch.float32).cuda() for n, v in filters.items()}
    tok, prob = fdllm.fdllm_sample(x.cuda(), torch.as_tensor(u, dtype=torch.float64).cuda(),
                                   mask_id=mask_id, **dev)
    return tok.cpu().tolist(), prob.cpu().double()


def _check(x, u, mask_id=-1, **filters):
    """Tokens equal; probabilities to float32's rounding, plus the weights'
    fixed-point steps (2^-45 each, at most 2^18 of them)."""
    tok, prob = _run(x, u, mask_id, **filters)
    for r in range(x.shape[0]):
        per = {n: float(torch.as_tensor(v, dtype=torch.float32)[r]) for n, v in filters.items() if v is not None}
        if "top_k" in per:
            per["top_k"] = int(filters["top_k"][r])
        want, p, _ = kv8_ref.sample_row(x[r].double().numpy(), u[r], mask_id=mask_id, **per)
        assert tok[r] == want, (r, tok[r], want, per)
        assert abs(prob[r] - p) <= 2.0 ** -23 * p + 2.0 ** -27, (r, prob[r], p)


def _logits(g, rows, vocab, spread=2.5):
    x = torch.randn(rows, vocab, generator=g) * spread
    x.scatter_add_(1, torch.randint(0, vocab, (rows, 8), generator=g), 6 * torch.rand(rows, 8, generator=g))
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 2), (5, 33), (3, 512), (7, 2051), (2, 30001), (2, 152064)])
@pytest.mark.parametrize("kind", ["plain", "k", "p", "minp", "all", "greedy"])
def test_sample(dtype, rows, vocab, kind):
    g = torch.Generator().manual_seed(rows * 7 + vocab)
    x = _logits(g, rows, vocab).to(TYPES[dtype])
    u = torch.rand(rows, generator=g, dtype=torch.float64).tolist()
    f = {"temperature": (0.4 + torch.rand(rows, generator=g)).tolist()}
    if kind in ("k", "all"):
        f["top_k"] = torch.randint(1, 60, (rows,), generator=g).tolist()
    if kind in ("p", "all"):
        f["top_p"] = (0.05 + 0.94 * torch.rand(rows, generator=g)).tolist()
    if kind in ("minp", "all"):
        f["min_p"] = (0.2 * torch.rand(rows, generator=g)).tolist()
    if kind == "greedy":
        f["temperature"] = [0.0 if r % 2 == 0 else -1.0 for r in range(rows)]
    _check(x, u, mask_id=vocab - 1 if vocab > 2 else -1, **f)


def test_rows_of_equal_logits():
    """Ties: the lower id counts as the heavier one; cuts fall inside a tie."""
    for vocab in (7, 1000, 40000):
        x = torch.full((6, vocab), 1.25)
        x[:, vocab // 2] = 1.25
        u = [0.0, 0.3, 0.5, 0.999, 0.7, 1 - 2.0 ** -53]
        _check(x, u)
        _check(x, u, top_k=[1, 2, 3, 4, 5, 6])
        _check(x, u, top_p=[0.1, 0.25, 0.5, 0.75, 0.9, 0.3])
        _check(x, u, top_p=[0.5] * 6, top_k=[3, 4, 5, 6, 7, 5], min_p=[1.0] * 6)
        y = x.clone()
        y[:, ::3] = 2.0
        _check(y, u, top_k=[vocab // 3 + 2] * 6)
        _check(y, u, top_p=[0.6, 0.7, 0.8, 0.9, 0.2, 0.45])
        _check(y, u, temperature=[0.0] * 6, mask_id=0)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_kept_sets(dtype):
    """Kept sets beyond what is gathered and sorted: flat rows, wide nuclei,
    large top_k, alone and together; heavy ties in 16-bit logits."""
    g = torch.Generator().manual_seed(21)
    x = (torch.randn(6, 60001, generator=g) * torch.tensor([0.01, 0.3, 1.0, 2.0, 4.0, 1.0])[:, None]).to(TYPES[dtype])
    u = torch.rand(6, generator=g, dtype=torch.float64).tolist()
    t = [1.0, 0.7, 1.3, 1.0, 1.0, 50.0]
    _check(x, u, temperature=t, top_p=[0.9, 0.5, 0.95, 0.99, 0.999, 0.3], mask_id=60000)
    _check(x, u, temperature=t, top_k=[2000, 4096, 5000, 1025, 30000, 59999])
    _check(x, u, temperature=t, top_k=[2000, 4096, 5000, 1500, 30000, 59999],
           top_p=[0.9, 0.5, 0.95, 0.99, 0.999, 0.3])
    _check(x, u, temperature=t, top_k=[700, 512, 300, 1000, 1024, 250], top_p=[0.5] * 6, min_p=[0.1] * 6)
    _check(x, u, temperature=t, min_p=[0.5, 0.01, 1e-3, 1e-4, 1e-6, 0.99])
    _check(x, u, temperature=t, top_p=[0.9, 0.5, 0.95, 0.99, 0.999, 0.3], min_p=[0.5, 0.01, 1e-3, 1e-4, 1e-6, 0.99])
    _check(x, u, temperature=[0.0] * 6, top_p=[0.7] * 6)


def test_many_rows_and_the_largest_vocabulary():
    g = torch.Generator().manual_seed(22)
    x = _logits(g, 700, 2051, 1.5)
    u = torch.rand(700, generator=g, dtype=torch.float64).tolist()
    _check(x, u, top_p=[0.8] * 700, top_k=[100] * 700, mask_id=17)
    for dtype in TYPES.values():
        y = _logits(g, 2, 1 << 18, 1.5).to(dtype)
        _check(y, [0.3, 0.9], top_p=[0.9, 0.2])
        _check(y, [0.3, 0.9])


@pytest.mark.parametrize("dtype", TYPES)
def test_many_long_rows(dtype):
    """So many long rows that they are not copied on chip: an odd vocabulary in
    a wider buffer, rows without a live token, with infinities, NaN and ties, and
    kept sets of every size."""
    rows, vocab = 300, 41003
    g = torch.Generator().manual_seed(31)
    x = torch.full((rows, 41008), float("nan"))
    x[:, :vocab] = _logits(g, rows, vocab, 1.5) * torch.tensor([0.01, 0.5, 1.0, 2.0])[torch.arange(rows) % 4, None]
    x[5] = -float("inf")
    x[6, 3:vocab:11] = float("inf")
    x[7, :vocab] = 0.5
    x[8, ::2] = float("nan")
    x[9, :vocab] = -float("inf")
    x[9, vocab - 1] = 7.0
    x = x.to(TYPES[dtype])
    u = torch.rand(rows, generator=g, dtype=torch.float64)
    pick = torch.randint(0, 1 << 30, (4, rows), generator=g)
    f = {"temperature": torch.where(pick[0] % 5 == 0, 0.0, 0.3 + (pick[0] % 1000) / 800.0),
         "top_k": torch.where(pick[1] % 2 == 0, 0, 1 + pick[1] % 3001).to(torch.int32),
         "top_p": torch.where(pick[2] % 2 == 0, 1.0, 0.05 + (pick[2] % 997) / 1050.0),
         "min_p": torch.where(pick[3] % 2 == 0, 0.0, (pick[3] % 991) / 5000.0)}
    f = {n: v.to(torch.int32 if n == "top_k" else torch.float32) for n, v in f.items()}
    mask = vocab - 1
    tok, prob = fdllm.fdllm_sample(x.cuda()[:, :vocab], u.cuda(), mask_id=mask, **{n: v.cuda() for n, v in f.items()})
    for r in range(rows):
        want, p, _ = kv8_ref.sample_row(x[r, :vocab].double().numpy(), float(u[r]), mask_id=mask,
                                        **{n: (int if n == "top_k" else float)(v[r]) for n, v in f.items()})
        assert int(tok[r]) == want, r
        assert abs(float(prob[r]) - p) <= 2.0 ** -23 * p + 2.0 ** -27, r


def test_filter_settings_at_their_ends():
    g = torch.Generator().manual_seed(2)
    x = _logits(g, 8, 700)
    u = torch.rand(8, generator=g, dtype=torch.float64).tolist()
    _check(x, u, top_k=[0, -5, 1, 699, 700, 701, 2 ** 31 - 1, -2 ** 31])
    _check(x, u, top_p=[0.0, -1.0, 1.0, 2.0, 1e-30, 1 - 2.0 ** -24, 0.5, float("inf")])
    _check(x, u, min_p=[0.0, -1.0, 1.0, 2.0, 1e-30, 0.999, 0.5, float("inf")])
    _check(x, u, temperature=[1e-30, 1e30, float("inf"), 1e-3, 100.0, -0.0, float("nan"), 1.0])
    _check(x, [0.0, 1 - 2.0 ** -53, 1.0, 1.5, -0.5, 0.5, 0.25, 0.75])


def test_infinities_nan_and_empty_rows():
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[-inf, nan, -inf, -inf], [-inf, nan, 3.0, -inf], [inf, 0.0, inf, nan],
                      [0.0, -0.0, -inf, 0.0], [-3e38, 3e38, nan, 0.0], [-inf, -inf, -inf, 5.0]])
    for k in (None, [2] * 6):
        for p in (None, [0.6] * 6):
            for t in (None, [0.0] * 6, [1e30] * 6):
                _check(x, [0.1, 0.2, 0.7, 0.4, 0.5, 0.5], top_k=k, top_p=p, temperature=t)
                _check(x, [0.1, 0.2, 0.7, 0.4, 0.5, 0.5], mask_id=3, top_k=k, top_p=p, temperature=t)
    assert _run(x, [0.1] * 6, mask_id=3)[0][5] == -1


def test_strides_alignment_and_defaults():
    """Rows of a wider buffer whose start is aligned to an element only."""
    g = torch.Generator().manual_seed(3)
    for dtype in TYPES.values():
        wide = _logits(g, 5, 1107).to(dtype)
        x = wide[:, 3:1004]
        u = torch.rand(5, generator=g, dtype=torch.float64).tolist()
        tok, _ = fdllm.fdllm_sample(wide.cuda()[:, 3:1004], torch.tensor(u, dtype=torch.float64).cuda())
        assert tok.tolist() == [kv8_ref.sample_row(x[r].double().numpy(), u[r])[0] for r in range(5)]
    tok, prob = fdllm.fdllm_sample(torch.zeros(0, 9, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda"))
    assert tok.numel() == 0 and prob.numel() == 0


def test_confidence_is_the_decoders():
    """A greedy row without filters: the softmax probability of the argmax
    with the mask id excluded, the decoder's confidence."""
    g = torch.Generator().manual_seed(4)
    x = 3 * torch.randn(16, 2051, generator=g)
    tok, prob = _run(x, [0.5] * 16, mask_id=2050, temperature=[0.0] * 16)
    z = x.double()
    z[:, 2050] = -float("inf")
    p = torch.softmax(z, -1)
    assert tok == p.argmax(-1).tolist()
    assert (prob - p.amax(-1)).abs().max() <= 2.0 ** -24


def test_frequencies_follow_the_distribution():
    """4096 evenly spread numbers draw every token as often as its share
    says, to one count at each of its two borders."""
    x = torch.tensor([[0.0, 1.0, 2.0, 0.5, -1.0]]).expand(4096, 5).contiguous()
    u = ((torch.arange(4096, dtype=torch.float64) + 0.5) / 4096).tolist()
    tok, _ = _run(x, u, temperature=[0.8] * 4096)
    count = np.bincount(tok, minlength=5)
    p = torch.softmax(x[0].double() / np.float32(0.8), -1).numpy()
    assert (np.abs(count - 4096 * p) <= 1.0).all()


def test_graph_and_repeatability():
    g = torch.Generator().manual_seed(5)
    x = _logits(g, 9, 50000).cuda()
    u = torch.rand(9, generator=g, dtype=torch.float64).cuda()
    p = torch.full((9,), 0.9, device="cuda")
    k = torch.full((9,), 500, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in fdllm.fdllm_sample(x, u, top_p=p, top_k=k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, prob = fdllm.fdllm_sample(x, u, top_p=p, top_k=k)
    for _ in range(4):
        tok.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, want[0]) and torch.equal(prob, want[1])
