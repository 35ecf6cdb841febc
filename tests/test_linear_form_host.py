"""MOE_LINEAR_FORM, the switch that forces the form of moe_linear's products: names that it does not have, and forms that
do not fit the call, are refused before any CUDA call."""
import pytest

FAKE = 1 << 20  # 16-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


def forward(M, rows):
    return M.lib.moe_linear(FAKE, FAKE, None, 0, None, 0, rows, 256, 128, 0, None, FAKE, 0, None)


def backward(M, rows, dx=FAKE, dw=FAKE, db=None):
    return M.lib.moe_linear_backward(FAKE, 0, None, FAKE, FAKE, rows, 256, 128, 0, dx, dw, 0, db, FAKE, 1 << 30, None)


@pytest.mark.parametrize("name", ["fast", "p", "pairs", "Split", "tokens", " pair", "1", "x" * 40])
@pytest.mark.parametrize("rows", [1, 4])
def test_unknown_names_are_refused(M, monkeypatch, name, rows):
    monkeypatch.setenv("MOE_LINEAR_FORM", name)
    n = M.lib.moe_launch_count()
    for call in (forward, backward):
        assert call(M, rows) == 1
        assert "MOE_LINEAR_FORM" in M.last_error() and name[:32] in M.last_error()
    assert backward(M, rows, dx=None, dw=None, db=FAKE) == 1
    assert M.lib.moe_launch_count() == n


def test_the_one_token_form_is_refused_where_it_does_not_fit(M, monkeypatch):
    monkeypatch.setenv("MOE_LINEAR_FORM", "token")
    for call in (lambda: forward(M, 4), lambda: forward(M, 2), lambda: backward(M, 1), lambda: backward(M, 4),
                 lambda: backward(M, 1, dx=None)):
        assert call() == 1 and "MOE_LINEAR_FORM=token" in M.last_error()


def test_no_rows_need_no_form(M, monkeypatch):
    monkeypatch.setenv("MOE_LINEAR_FORM", "fast")
    assert forward(M, 0) == 0


@pytest.mark.gpu
def test_forms_of_one_row(M, monkeypatch):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((1, 520), (264, 520)))
    ref, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    got = {}
    for name in (None, "", "token", "split", "pair"):
        if name is None:
            monkeypatch.delenv("MOE_LINEAR_FORM", raising=False)
        else:
            monkeypatch.setenv("MOE_LINEAR_FORM", name)
        got[name] = torch.empty((1, 264), device="cuda")
        M.moe_linear(x, w, got[name])
        # sums of 520 products, each addition off by at most 2^-23 of the running sum, 16 products at a time
        assert ((got[name].double() - ref).abs() <= 2.0 ** -23 * (520 / 16 + 4) * size).all()
    assert torch.equal(got[None], got[""]) and torch.equal(got[None], got["token"])
