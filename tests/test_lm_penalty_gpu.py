"""GPU: logits penalties against their fp64 definition, element by element;
untouched logits bit for bit."""
import pytest
import torch

import lm_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


def make(rows, V, L, nb, masks, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    c = dict(logits=(3 * torch.randn(rows, V, generator=g)).to(DT[dt]),
             tokens=(torch.exp(r(rows, L) * torch.log(torch.tensor(float(V)))) - 1).clamp(0, V - 1).int(),
             lens=torch.randint(0, L + 1, (rows,), generator=g).int(),
             rep=1 + 0.5 * r(rows), freq=0.3 * r(rows), pres=r(rows),
             bias_ids=None, bias=None, mask=None, mask_index=None)
    c["lens"][0] = L
    c["prompt"] = (c["lens"] * r(rows)).int()
    if nb:
        c["bias_ids"] = torch.stack([torch.randperm(V, generator=g)[:nb] if nb <= V else
                                     torch.randint(0, V, (nb,), generator=g)
                                     for _ in range(rows)]).int()
        c["bias_ids"][:, ::5] = -1
        c["bias"] = 4 * torch.randn(rows, nb, generator=g)
    if masks:
        c["mask"] = torch.randint(-2**31, 2**31, (masks, (V + 31) // 32), generator=g).int()
        c["mask"][0] = 0               # leaves nothing
        c["mask_index"] = torch.randint(-1, masks, (rows,), generator=g).int()
        c["mask_index"][0] = 0
    return c


def run(lm, c, what="", in_place=False):
    rows, V = c["logits"].shape
    what += f" rows={rows} V={V} L={0 if c['tokens'] is None else c['tokens'].shape[1]} {c['logits'].dtype}"
    print(what, flush=True)
    cu = {k: None if v is None else v.cuda() for k, v in c.items()}
    p = lm.LogitsPenalty(V)
    ws = p.workspace(rows)
    x = cu["logits"].clone()
    out = x if in_place else torch.full_like(x, 7.0)
    p.apply(x, out, tokens=cu["tokens"], prompt_lens=cu["prompt"], lens=cu["lens"],
            repetition=cu["rep"], frequency=cu["freq"], presence=cu["pres"],
            bias_ids=cu["bias_ids"], bias_values=cu["bias"], mask=cu["mask"],
            mask_index=cu["mask_index"], workspace=ws)
    want = ref.penalty(c["logits"], c["tokens"], c["prompt"], c["lens"], c["rep"], c["freq"],
                       c["pres"], c["bias_ids"], c["bias"], c["mask"], c["mask_index"])
    ref.check(dict(out=out), want, what)
    same = want["out"][0] == c["logits"].double()
    assert torch.equal(out.cpu()[same], c["logits"][same])
    return p.device_status(ws)


@pytest.mark.parametrize("V", [1, 7, 8, 31, 33, 1000, 1023, 1024, 1025, 4097, 20011])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_vocabularies(lm, V, dt):
    assert run(lm, make(3, V, 50, min(9, V), 3, dt)) == "SGB_OK"
    assert run(lm, make(3, V, 50, min(9, V), 3, dt, seed=1), in_place=True) == "SGB_OK"


@pytest.mark.parametrize("L", [1, 2, 3, 4, 5, 255, 2047, 5000])
def test_lengths(lm, L):
    run(lm, make(4, 3000, L, 0, 0, "f32"))


@pytest.mark.parametrize("rows,V", [(600, 900), (130, 9000), (40, 40000)])
def test_slices(lm, rows, V):
    # rows and widths that give every slice size up to the largest
    run(lm, make(rows, V, 40, 5, 4, "bf16"))


@pytest.mark.parametrize("nb", [1, 300, 1023])
def test_biases(lm, nb):
    run(lm, make(3, 2500, 30, nb, 0, "f32"))


def test_repeated_biases_add_up(lm):
    c = make(3, 2500, 30, 40, 2, "f32")
    c["bias_ids"][1, 3:9] = 77
    c["bias_ids"][2, 1] = c["bias_ids"][2, 2]
    run(lm, c, "repeated biases")


def test_without_any(lm):
    c = make(3, 1500, 20, 0, 0, "f16")
    for k in ("tokens", "lens", "prompt", "rep", "freq", "pres"):
        c[k] = None
    assert run(lm, c, "nothing") == "SGB_OK"


def test_each_alone(lm):
    for drop in (("rep",), ("freq",), ("pres",), ("prompt",), ("lens", "prompt"),
                 ("rep", "freq", "pres")):
        c = make(3, 1500, 60, 0, 0, "f32")
        for k in drop:
            c[k] = None
        run(lm, c, f"without {drop}")


def test_a_mask_for_every_row(lm):
    c = make(4, 1300, 20, 0, 4, "bf16")
    c["mask_index"] = None
    run(lm, c, "own masks")


def test_infinite_and_nan_logits(lm):
    c = make(2, 1200, 300, 0, 0, "f32")
    c["logits"][0, :20] = -torch.inf
    c["logits"][0, 20:25] = torch.inf
    c["logits"][1, :9] = torch.finfo(torch.float32).min
    c["logits"][1, 9:12] = torch.nan
    run(lm, c, "infinities")


def test_one_token_over_and_over(lm):
    c = make(2, 5000, 70000, 0, 0, "f32")
    c["tokens"][0] = 4321
    c["lens"][:] = 70000
    c["prompt"][0] = 5
    c["freq"][0] = 1e-3
    c["lens"][1] = c["prompt"][1] = 3
    run(lm, c, "counts past 16 bits")


def test_bad_contents_are_reported_and_left_out(lm):
    c = make(4, 900, 20, 4, 2, "f32")
    c["tokens"][0, 3] = -1          # row 0 uses its whole length
    assert run(lm, c, "negative token") == "SGB_OK"
    c["tokens"][0, 5] = 900
    assert run(lm, c, "token past the vocabulary") == "SGB_ERR_INDEX_OUT_OF_RANGE"
    c["tokens"][0, 5] = 2**31 - 1
    assert run(lm, c, "token far past it") == "SGB_ERR_INDEX_OUT_OF_RANGE"
    c = make(4, 900, 20, 4, 2, "f32")
    c["bias_ids"][2, 1] = 900
    assert run(lm, c, "bias id") == "SGB_ERR_INDEX_OUT_OF_RANGE"
    c = make(4, 900, 20, 4, 2, "f32")
    c["mask_index"][3] = 2
    assert run(lm, c, "mask index") == "SGB_ERR_INDEX_OUT_OF_RANGE"
    c = make(4, 900, 20, 4, 2, "f32")
    lens = c["lens"].clone()
    lens[2] = 20
    c["prompt"][2] = 20
    p = lm.LogitsPenalty(900)
    cu = {k: None if v is None else v.cuda() for k, v in c.items()}
    outs = []
    for bad in (False, True):
        n, m = lens.clone(), c["prompt"].clone()
        if bad:
            n[2], m[2] = 21, 25
        ws, out = p.workspace(4), torch.empty_like(cu["logits"])
        p.apply(cu["logits"], out, tokens=cu["tokens"], prompt_lens=m.cuda(), lens=n.cuda(),
                repetition=cu["rep"], workspace=ws)
        outs.append(out)
        assert p.device_status(ws) == ("SGB_ERR_BAD_OFFSETS" if bad else "SGB_OK")
    assert torch.equal(*outs)


def test_strides(lm):
    rows, V, L = 5, 1003, 33
    c = make(rows, V, L, 6, 3, "f16")
    cu = {k: None if v is None else v.cuda() for k, v in c.items()}
    p = lm.LogitsPenalty(V)
    ws, out = p.workspace(rows), torch.empty_like(cu["logits"])

    def wide(t, at, W):
        w = torch.full((t.shape[0], W), 3, dtype=t.dtype, device="cuda")
        w[:, at:at + t.shape[1]] = t
        return w, w[:, at:at + t.shape[1]]
    kw = dict(prompt_lens=cu["prompt"], lens=cu["lens"], repetition=cu["rep"],
              frequency=cu["freq"], presence=cu["pres"], mask_index=cu["mask_index"], workspace=ws)
    p.apply(cu["logits"], out, tokens=cu["tokens"], bias_ids=cu["bias_ids"],
            bias_values=cu["bias"], mask=cu["mask"], **kw)
    wo, o = wide(torch.zeros_like(out), 7, 1111)
    p.apply(wide(cu["logits"], 1, 1100)[1], o, tokens=wide(cu["tokens"], 3, 41)[1],
            bias_ids=wide(cu["bias_ids"], 1, 9)[1], bias_values=wide(cu["bias"], 2, 10)[1],
            mask=wide(cu["mask"], 0, 40)[0], **kw)
    assert torch.equal(o, out)
    assert bool((wo[:, :7] == 3).all()) and bool((wo[:, 7 + V:] == 3).all())


@pytest.mark.parametrize("L", [8191, 8192, 8193, 16385, 40001])
def test_long_sequences(lm, L):
    """Either side of what one round of token loads holds."""
    c = make(2, 1500, L, 3, 0, "bf16")
    c["lens"][1] = L - 1
    c["prompt"][1] = L // 2
    run(lm, c, "long")


@pytest.mark.parametrize("V", [8193, 8199, 16385, 24571])
def test_last_slices(lm, V):
    """A last slice of one logit, of seven, of whole vectors and a part."""
    assert run(lm, make(300, V, 12, 4, 3, "f16"), in_place=True) == "SGB_OK"
