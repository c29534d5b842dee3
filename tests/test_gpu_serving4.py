"""The serving layer with prepared rows and with a cache in 4 bits: prefix, admission,
tokens, and the rows handed on to states."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("bits", [None, 4])
def test_layer_with_prepared_rows(cuda_device, dtype, prefix, bits):
    import torch
    import attn_reference as ref
    import kv4_reference as ref4
    from streaming_nystr_landmark_gb300 import nys, serving
    dt = getattr(torch, dtype)
    heads, kv, d, dv, page, tokens = 8, 2, 64, 128, 16, 3
    lens = [1, 40, 16, 0, 129]
    g = torch.Generator(device=cuda_device).manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device).to(dt)
    w = [1 + 0.1 * torch.randn(d, generator=g, device=cuda_device) for _ in range(2)]
    prep = nys.QKPrepare(heads, kv, d, dtype=dt, q_weight=w[0], k_weight=w[1],
                         rotation=nys.Rotation(d, base=1e6, device=cuda_device), device=cuda_device)
    layer = serving.ExactLayer(heads, kv, d, dv, len(lens), 64, page, 160, dtype=dt, device=cuda_device,
                               prepare=prep, bits=bits)
    pk, pv = rn(prefix, kv, d), rn(prefix, kv, dv)
    pos = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    if prefix:
        layer.set_prefix(pk, pv)
        with pytest.raises(ValueError, match="first request"):
            layer.set_prefix(pk, pv)
        pk = prep.rows(None, pk.clone(), pos(*range(prefix)))[1]
    q, k, v = rn(sum(lens), heads, d), rn(sum(lens), kv, d), rn(sum(lens), kv, dv)
    kept = q.clone(), k.clone()
    out = layer.admit(q, k, v, lens)
    assert torch.equal(q, kept[0]) and torch.equal(k, kept[1])
    at = pos(*[prefix + j for x in lens for j in range(x)])
    q, k = prep.rows(q, k, at)
    # Prompts are attended over their own rows as they are.
    ks = [torch.cat([pk, x]) for x in k.split(lens)]
    vs = [torch.cat([pv, x]) for x in v.split(lens)]
    want, _, bound, _ = ref.prompt(q, torch.cat(ks), torch.cat(vs), lens, [prefix + x for x in lens],
                                   heads // kv, 1 / math.sqrt(d), dt)
    extra = 0.0 if dt == torch.float32 else 2 * ref.EPS[dt] * float(torch.cat(vs).abs().max())
    ref.check(out, want, 2 * bound + extra + 2.0 ** -22, "prompts")
    own_k, own_v = list(k.split(lens)), list(v.split(lens))
    for n in range(tokens):
        q1, k1, v1 = rn(len(lens), heads, d), rn(len(lens), kv, d), rn(len(lens), kv, dv)
        out = layer.decode(q1, k1, v1)
        q1, k1 = prep.rows(q1, k1, pos(*[prefix + x + n for x in lens]))
        own_k = [torch.cat([a, b[None]]) for a, b in zip(own_k, k1)]
        own_v = [torch.cat([a, b[None]]) for a, b in zip(own_v, v1)]
        if bits is None:
            for i in range(len(lens)):
                a, b = layer.cached(i)
                assert torch.equal(a, own_k[i]) and torch.equal(b, own_v[i])
            want, _, bound, _ = ref.prompt(
                q1, torch.cat([x for y in own_k for x in (pk, y)]), torch.cat([x for y in own_v for x in (pv, y)]),
                [1] * len(lens), [prefix + len(x) for x in own_k], heads // kv, 1 / math.sqrt(d), dt)
            ref.check(out, want, bound, "token")
            continue
        # Over the values that the cache holds, in the prefix as they are.
        (kc, ks4, km), (vc, vs4, vm) = ref4.unpack(layer.cache.data, kv, d, dv, page)
        table = layer.table.long().cpu()
        for i, x in enumerate(own_k):
            j = torch.arange(len(x))
            s = table[i][j // page] * page + j % page
            hk, hv = ref4.values(kc[s], ks4[s], km[s]), ref4.values(vc[s], vs4[s], vm[s])
            step = ks4[s].double().repeat_interleave(64, -1)[..., :d]
            # (The rows here were rounded to their type; the codes come from before that.)
            near = step / 2 + (x.double().cpu().abs() + 1) * ref4.EPS[dt] * 2
            assert bool(((hk - x.double().cpu()).abs() <= near).all())
            a, b = layer.cached(i)
            assert torch.equal(a.cpu(), hk.float().to(dt)) and torch.equal(b.cpu(), hv.float().to(dt))
            ak = torch.cat([pk.double().cpu(), hk])
            av = torch.cat([pv.double().cpu(), hv])
            want, lse, bound = ref4.attend(q1[i], ak, av, 1 / math.sqrt(d), dt)
            # The prefix's result is rounded to its type, its weights too, before the join.
            size = av.abs().amax((0, 2)).repeat_interleave(heads // kv)[:, None]
            ref4.check(out[i], want, bound + 4 * ref4.EPS[dt] * size * (prefix > 0), f"token of request {i}")
    assert layer.status() == 0
    assert layer.lens.tolist() == [x + tokens for x in lens]


def test_states_are_sealed_on_a_4_bit_cache(cuda_device):
    """A request's rows, read back, seal landmark states that decode as those of the same
    values do."""
    import torch
    from streaming_nystr_landmark_gb300 import nys, serving
    heads, kv, d, t = 4, 2, 64, 96
    g = torch.Generator(device=cuda_device).manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device)
    layer = serving.ExactLayer(heads, kv, d, d, 1, 8, 16, 112, device=cuda_device, bits=4)
    q, k, v = rn(t, heads, d), rn(t, kv, d), rn(t, kv, d)
    layer.admit(q, k, v, [t])
    hk, hv = layer.cached(0)
    assert float((hk - k).abs().max()) < 0.4 and float((hv - v).abs().max()) < 0.4
    outs = []
    for a, b in ((hk, hv), (hk.clone(), hv.clone())):
        st = nys.NystromStates(m=8, w=16, sink=4, heads_per_kv=heads // kv, d=d, dv=d, n_groups=kv, device=cuda_device)
        serving.seal_prompts(st, q, a, b, [t])
        out = torch.empty((kv, heads // kv, d), device=cuda_device)
        st.step(q[0].view(kv, heads // kv, d).contiguous(), k[0].contiguous(), v[0].contiguous(), out)
        outs.append(out)
        st.close()
    assert torch.equal(*outs) and bool(outs[0].isfinite().all())


def test_layer_refusals(cuda_device):
    import torch
    from streaming_nystr_landmark_gb300 import nys, serving
    dev = cuda_device
    with pytest.raises(ValueError):
        serving.ExactLayer(4, 2, 64, 64, 1, 4, 16, 32, device=dev, bits=8)
    with pytest.raises(ValueError):
        serving.ExactLayer(4, 2, 64, 64, 1, 4, 8, 32, device=dev, bits=4)
    for bad in (nys.QKPrepare(4, 4, 64, device=dev), nys.QKPrepare(4, 2, 32, device=dev),
                nys.QKPrepare(4, 2, 64, dtype=torch.float16, device=dev)):
        with pytest.raises(ValueError):
            serving.ExactLayer(4, 2, 64, 64, 1, 4, 16, 32, device=dev, prepare=bad)
