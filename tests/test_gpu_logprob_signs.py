"""Log probabilities are at most 0 and entropies at least 0, whatever order a row's entries come in."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 7, 4099, 60000])
def test_signs_near_a_probability_of_one(V, dtype, n):
    # one entry above the others by just under, at and behind the lag of a row's reference (8 in
    # units of log 2) and far above it, before, among and behind them
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    steps = [5.5, 5.54, 5.545, 5.546, 5.55, 5.6, 11.0, 16.0, 17.0, 20.0, 30.0, 100.0]
    x, ids = [], []
    for low in (-1e4, 0.0):
        for step in steps:
            for at in sorted({0, n // 3, n // 2, n - 1}):
                row = torch.full((n,), low, device="cuda")
                row[torch.randint(0, n, (1,), generator=g, device="cuda")] = 0.0      # what a reference may begin with
                row[at] = step
                x.append(row)
                ids.append(at)
    x, ids = torch.stack(x).to(dtype), torch.tensor(ids, dtype=torch.int32, device="cuda")
    for T in (1.0, 0.7, 0.01):
        got = V.logprobs(x, ids, T=T, top=3)
        assert V.get_error() == 0
        assert (got.logprob <= 0).all() and (got.entropy >= 0).all() and (got.top_logprobs <= 0).all()
        lp = (x.double() / T).log_softmax(1)
        want = lp.gather(1, ids[:, None].long())[:, 0]
        # log2 of the sum and the distance, up to 2^9 beside it, in 32 bits: 16 roundings of both
        assert ((got.logprob - want).abs() <= 2.0 ** -20 * (1 + want.abs()) + 2.0 ** -20).all()
