"""What the two 8-bit parts of a query element and of a probability hold (as sfa_cache8_attn documents), on CPU."""

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def parts(x, k):
    """hi + lo / 2^k with hi = e4m3(x), lo = e4m3((x - hi) 2^k), in 64 bits."""
    r = lambda y: y.float().to(E4M3).double()  # noqa: E731
    hi = r(x)
    return hi + r((x - hi) * 2.0 ** k) / 2.0 ** k


def test_query_parts():
    """Every bf16 magnitude up to every largest element in (224, 448], as rows are scaled."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    x = (bits << 16).view(torch.float32).double()
    x = x[x <= 448.0]
    err = (parts(x, 4) - x).abs()
    assert float(x.max()) == 448.0
    for top in x[x > 224.0].tolist():
        own = x <= top
        assert torch.all(err[own & (x >= 2.0 ** -13 * top)] == 0)
        assert torch.all(err[own] <= 2.0 ** -21 * top)


def test_probability_parts():
    """Probabilities of every magnitude against their block's largest, which is scaled to 256."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(np.concatenate([256.0 * np.exp2(-rng.uniform(0, 40, 400000)), rng.uniform(0, 256, 400000), [256.0, 0.0]]))
    x = x.float().double()
    err = (parts(x, 5) - x).abs()
    assert torch.all(err <= torch.maximum(x * 2.0 ** -9, torch.tensor(256.0 * 2.0 ** -23, dtype=torch.float64)))
    assert parts(x[-2:], 5).tolist() == [256.0, 0.0]


def test_compact_keys_are_exact_down_to_small_scales():
    v = torch.arange(256, dtype=torch.uint8).view(E4M3).double()
    v = v[torch.isfinite(v)]
    for e in (-124, -60, 0, 100):
        assert torch.equal((v * 2.0 ** e).float().to(torch.bfloat16).double(), v * 2.0 ** e)
    assert not torch.equal((v * 2.0 ** -126).float().to(torch.bfloat16).double(), v * 2.0 ** -126)
