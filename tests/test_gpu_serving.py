"""The exact operators together, as a serving loop uses them: a shared prefix,
prompts admitted in one packed batch, tokens decoded one by one, and landmark
states sealed on the same prompts."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("prefix", [0, 37])
def test_layer_serves_prompts_and_tokens(cuda_device, dtype, prefix):
    import torch
    import attn_reference as ref
    from streaming_nystr_landmark_gb300 import serving
    dt = getattr(torch, dtype)
    heads, kv, d, dv, page, tokens = 8, 2, 64, 128, 16, 6
    lens = [1, 40, 16, 0, 129]
    g = torch.Generator(device=cuda_device).manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device).to(dt)
    layer = serving.ExactLayer(heads, kv, d, dv, len(lens), 64, page, 160, dtype=dt,
                               device=cuda_device)
    pk, pv = rn(prefix, kv, d), rn(prefix, kv, dv)
    if prefix:
        layer.set_prefix(pk, pv)
    q, k, v = rn(sum(lens), heads, d), rn(sum(lens), kv, d), rn(sum(lens), kv, dv)
    out = layer.admit(q, k, v, lens)
    # Plain form: every request's keys are the prefix's and its own.
    ks = [torch.cat([pk, x]) for x in k.split(lens)]
    vs = [torch.cat([pv, x]) for x in v.split(lens)]
    want, _, bound, _ = ref.prompt(q, torch.cat(ks), torch.cat(vs), lens,
                                   [prefix + x for x in lens], heads // kv, 1 / math.sqrt(d), dt)
    # Two results are rounded to their type and weighed before the last rounding.
    extra = 0.0 if dt == torch.float32 else 2 * ref.EPS[dt] * float(torch.cat(vs).abs().max())
    ref.check(out, want, 2 * bound + extra + 2.0 ** -22, "prompts")
    for _ in range(tokens):
        q1, k1, v1 = rn(len(lens), heads, d), rn(len(lens), kv, d), rn(len(lens), kv, dv)
        out = layer.decode(q1, k1, v1)
        ks = [torch.cat([a, b[None]]) for a, b in zip(ks, k1)]
        vs = [torch.cat([a, b[None]]) for a, b in zip(vs, v1)]
        want, _, bound, _ = ref.prompt(q1, torch.cat(ks), torch.cat(vs), [1] * len(lens),
                                       [len(x) for x in ks], heads // kv, 1 / math.sqrt(d), dt)
        ref.check(out, want, bound, "token")
    assert layer.attention.status() == 0
    assert layer.lens.tolist() == [x + tokens for x in lens]


def test_layer_refuses_what_does_not_fit(cuda_device):
    import torch
    from streaming_nystr_landmark_gb300 import serving
    layer = serving.ExactLayer(2, 2, 64, 64, 2, 4, 8, 16, dtype=torch.bfloat16, device=cuda_device)
    z = lambda n, h: torch.zeros((n, h, 64), dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError, match="outgrow"):
        layer.admit(z(20, 2), z(20, 2), z(20, 2), [3, 17])
    layer.admit(z(24, 2), z(24, 2), z(24, 2), [8, 16])
    with pytest.raises(ValueError, match="pages"):
        serving.ExactLayer(2, 2, 64, 64, 2, 2, 8, 16, dtype=torch.bfloat16,
                           device=cuda_device).admit(z(24, 2), z(24, 2), z(24, 2), [8, 16])
    with pytest.raises(ValueError, match="first token"):
        layer.admit(z(2, 2), z(2, 2), z(2, 2), [1, 1])
    with pytest.raises(ValueError, match="before"):
        layer.set_prefix(z(2, 2), z(2, 2))


def test_layer_refuses_rows_and_lengths_that_differ(cuda_device):
    import torch
    from streaming_nystr_landmark_gb300 import serving
    layer = serving.ExactLayer(4, 2, 64, 64, 2, 8, 16, 64, device=cuda_device)
    z = lambda n, h: torch.zeros(n, h, 64, device=cuda_device)
    with pytest.raises(ValueError, match="pages wanted"):
        layer.set_prefix(z(130, 2), z(130, 2))      # 9 pages of a pool of 8
    with pytest.raises(ValueError, match="lengths"):
        layer.admit(z(5, 4), z(5, 2), z(5, 2), [5])
    with pytest.raises(ValueError, match="lengths"):
        layer.admit(z(5, 4), z(5, 2), z(5, 2), [6, -1])
    with pytest.raises(ValueError, match="rows"):
        layer.admit(z(5, 4), z(5, 2), z(5, 2), [5, 1])
    with pytest.raises(ValueError, match="one row"):
        layer.decode(z(1, 4), z(1, 2), z(1, 2))
    # Nothing was taken or counted by any of them.
    assert layer.used == 0 and layer.lengths == [0, 0] and layer.prefix_len == 0
    layer.admit(z(6, 4), z(6, 2), z(6, 2), [5, 1])
    assert layer.lengths == [5, 1] and layer.lens.tolist() == [5, 1]


def _state(layer):
    return (layer.used, list(layer.lengths), layer.lens.tolist(), layer.prefix_len,
            layer.prefix_pages is None, layer.table.tolist())


def test_layer_refuses_tensors_before_anything_is_counted(cuda_device, monkeypatch):
    """Tensors of another type, geometry or layout, and memory that is not there,
    leave the layer as it was: the right call made next succeeds."""
    import torch
    import attn_reference as ref
    from streaming_nystr_landmark_gb300 import serving
    heads, kv, d, dv = 4, 2, 64, 32
    layer = serving.ExactLayer(heads, kv, d, dv, 2, 16, 16, 64, device=cuda_device)
    g = torch.Generator(device=cuda_device).manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device)

    def refused(call, q, k, v, *more):
        """Every tensor wrong in every way, one at a time."""
        good, names = [q, k, v], ("q", "k", "v")
        bad = {"type": lambda t: t.bfloat16(), "host": lambda t: t.cpu(),
               "heads": lambda t: torch.cat([t, t], 1), "dim": lambda t: torch.cat([t, t], 2),
               "layout": lambda t: t.transpose(1, 2).contiguous().transpose(1, 2),
               "rows": lambda t: t[:-1]}
        for i, name in enumerate(names):
            if good[i] is None:
                continue
            for why, change in bad.items():
                args = list(good)
                args[i] = change(good[i])
                before = _state(layer)
                with pytest.raises(ValueError):
                    call(*[a for a in args if a is not None], *more)
                assert _state(layer) == before, (name, why)

        def no_memory(*a, **kw):
            raise torch.cuda.OutOfMemoryError("out of memory")
        if q is not None:
            before = _state(layer)
            with monkeypatch.context() as m:
                m.setattr(torch, "empty", no_memory)
                with pytest.raises(torch.cuda.OutOfMemoryError):
                    call(q, k, v, *more)
            assert _state(layer) == before

    pk, pv = rn(20, kv, d), rn(20, kv, dv)
    refused(layer.set_prefix, None, pk, pv)
    layer.set_prefix(pk, pv)
    lens = [5, 30]
    q, k, v = rn(35, heads, d), rn(35, kv, d), rn(35, kv, dv)
    refused(layer.admit, q, k, v, lens)
    layer.admit(q, k, v, lens)
    q1, k1, v1 = rn(2, heads, d), rn(2, kv, d), rn(2, kv, dv)
    refused(layer.decode, q1, k1, v1)
    out = layer.decode(q1, k1, v1)
    ks = [torch.cat([pk, a, b[None]]) for a, b in zip(k.split(lens), k1)]
    vs = [torch.cat([pv, a, b[None]]) for a, b in zip(v.split(lens), v1)]
    want, _, bound, _ = ref.prompt(q1, torch.cat(ks), torch.cat(vs), [1, 1],
                                   [len(x) for x in ks], heads // kv, 1 / math.sqrt(d), torch.float32)
    ref.check(out, want, bound, "token")
    assert layer.lengths == [6, 31] and layer.lens.tolist() == [6, 31]


def test_layer_reports_what_its_calls_met(cuda_device):
    """Bits of the attention's calls and of every plan, also of one that was
    replaced since."""
    import torch
    from streaming_nystr_landmark_gb300 import nys, serving
    layer = serving.ExactLayer(4, 2, 64, 64, 2, 16, 16, 64, device=cuda_device)
    z = lambda n, h: torch.zeros(n, h, 64, device=cuda_device)
    layer.admit(z(9, 4), z(9, 2), z(9, 2), [5, 4])
    assert layer.status() == 0
    layer.table[1, 0] = -1
    layer._plan([0, 1])                 # the token's page is gone
    layer._plan([1, 1])                 # another size of plan
    assert layer.status() & nys.NYS_PLAN_NO_PAGES
    layer.clear_status()
    assert layer.status() == 0
    layer.table[1, 0] = 1 << 20
    layer.decode(z(2, 4), z(2, 2), z(2, 2))
    assert layer.status() & nys.NYS_ATTN_BAD_PAGE


def test_landmark_states_of_the_same_prompts(cuda_device):
    """seal_prompts seals exactly what nys_seal seals group by group."""
    import torch
    from streaming_nystr_landmark_gb300 import nys, serving
    heads, kv, d, lens = 4, 2, 64, [80, 131]
    m, w, sink = 8, 16, 4
    g = torch.Generator(device=cuda_device).manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda_device)
    q, k, v = rn(sum(lens), heads, d), rn(sum(lens), kv, d), rn(sum(lens), kv, d)
    geo = (m, w, sink, heads // kv, d, d, len(lens) * kv)
    both = nys.NystromStates(*geo, device=cuda_device)
    serving.seal_prompts(both, q, k, v, lens)
    each = nys.NystromStates(*geo, device=cuda_device)
    at = 0
    for i, t in enumerate(lens):
        cut = slice(at, at + t)
        qs = q[cut].view(t, kv, heads // kv, d).permute(1, 2, 0, 3).contiguous()
        each.seal(qs, k[cut].transpose(0, 1).contiguous(), v[cut].transpose(0, 1).contiguous(),
                  g0=i * kv, n=kv)
        at += t
    for name in ("win_k", "sink_v", "k_tilde", "q_tilde", "mu", "t_hat", "z_hat", "m_max", "far_len"):
        assert torch.equal(both.region(name), each.region(name)), name


def test_landmark_states_refuse_rows_without_a_length(cuda_device):
    """Rows past the lengths' sum would be left out of every state in silence."""
    import torch
    from streaming_nystr_landmark_gb300 import nys, serving
    q, k, v = (torch.zeros(200, h, 64, device=cuda_device) for h in (4, 2, 2))
    states = nys.NystromStates(8, 16, 4, 2, 64, 64, 4, device=cuda_device)
    for lens in ([80, 100], [80, 131]):
        with pytest.raises(ValueError, match="rows"):
            serving.seal_prompts(states, q, k, v, lens)
    with pytest.raises(ValueError, match="rows"):
        serving.seal_prompts(states, q, k, v[:-1], [80, 120])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_landmark_states_of_16_bit_prompts(cuda_device, dtype):
    """The same states as of the values in f32."""
    import torch
    from streaming_nystr_landmark_gb300 import nys, serving
    lens = [80, 131]
    g = torch.Generator(device=cuda_device).manual_seed(2)
    q, k, v = (torch.randn((sum(lens), h, 64), generator=g, device=cuda_device)
               .to(getattr(torch, dtype)) for h in (4, 2, 2))
    geo = (8, 16, 4, 2, 64, 64, 4)
    a, b = (nys.NystromStates(*geo, device=cuda_device) for _ in range(2))
    serving.seal_prompts(a, q, k, v, lens)
    serving.seal_prompts(b, q.float(), k.float(), v.float(), lens)
    for name in ("win_k", "sink_v", "k_tilde", "q_tilde", "t_hat", "z_hat"):
        assert torch.equal(a.region(name), b.region(name)), name
