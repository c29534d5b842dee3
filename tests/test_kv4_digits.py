"""kv4_digits' measure tells weights of 22 bits from weights of 11 and 8, on the CPU."""
import math

import pytest

torch = pytest.importorskip("torch")
kv4_digits = pytest.importorskip("kv4_digits")


@pytest.mark.parametrize("geo", [(16, 8, 128), (1, 1, 64), (8, 2, 256), (8, 1, 64)])
@pytest.mark.parametrize("keys", [2, 17, 300, 2000])
def test_fewer_bits_of_a_weight_are_seen(geo, keys):
    import kv4_reference as ref
    heads, kv, d = geo
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((keys, kv, d), generator=g) for _ in range(2))
    kc, vc = ref.quantize(k), ref.quantize(v)
    q = torch.randn((3, heads, d), generator=g)
    held = ref.values(*kc)
    worst = {f: 0.0 for f in (kv4_digits.two_f16, kv4_digits.one_f16, kv4_digits.bf16)}
    for x in q:
        want, _, _ = ref.attend(x, held, ref.values(*vc), 1 / math.sqrt(d), torch.float32)
        for f in worst:
            got = kv4_digits.attend(x, held, vc, 1 / math.sqrt(d), f)
            worst[f] = max(worst[f], kv4_digits.off(got, want))
    assert worst[kv4_digits.two_f16] <= kv4_digits.MOST / 4
    assert worst[kv4_digits.one_f16] > 4 * kv4_digits.MOST and worst[kv4_digits.bf16] > 4 * kv4_digits.MOST
