"""Refusals of the dense operators' Python calls that need no GPU: weights, gradients
and matrices of another shape with as many elements.  They come before anything
asks for a device."""
import pytest
import torch

BF = torch.bfloat16
T, D_, H_ = 6, 64, 128


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_expert_gemm_gb300 as m
    return m


def _ffn():
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)
    return dict(x=z(T, D_), w_gate=z(H_, D_), w_up=z(H_, D_), w_down=z(D_, H_), token_scale=None, h_act=z(T, H_),
                p_save=z(T, H_), q_save=z(T, H_), dy=z(T, D_), dx_in=None, dx=z(T, D_),
                dw_gate=z(H_, D_, dt=torch.float32), dw_up=z(H_, D_, dt=torch.float32),
                dw_down=z(D_, H_, dt=torch.float32), dtoken_scale=None, ws=torch.zeros(1 << 16, dtype=torch.uint8))


BAD = ["transposed", "flat", "split", "more"]


def _bad(t, how):
    rows, cols = t.shape[-2:]
    if how == "transposed":
        return torch.zeros(*t.shape[:-2], cols, rows, dtype=t.dtype)
    if how == "flat":
        return t.reshape(-1)
    if how == "split":
        return t.reshape(*t.shape[:-2], rows * 2, cols // 2)
    return torch.zeros(*t.shape[:-2], rows + 8, cols, dtype=t.dtype)


@pytest.mark.parametrize("how", BAD)
@pytest.mark.parametrize("name", ["w_gate", "w_up", "w_down"])
def test_gated_ffn_refuses_weights_of_another_shape(moe, name, how):
    a = _ffn()
    a[name] = _bad(a[name], how)
    with pytest.raises(ValueError, match="expected"):
        moe.gated_ffn(a["x"], a["w_gate"], a["w_up"], a["w_down"], None, None, a["dx"], a["h_act"], None, None, a["ws"])


@pytest.mark.parametrize("how", BAD)
@pytest.mark.parametrize("name", ["w_gate", "w_up", "w_down", "dw_gate", "dw_up", "dw_down"])
def test_gated_ffn_backward_refuses_matrices_of_another_shape(moe, name, how):
    a = _ffn()
    a[name] = _bad(a[name], how)
    with pytest.raises(ValueError, match="expected"):
        moe.gated_ffn_backward(*a.values())


def test_gated_ffn_names_the_tensor(moe):
    a = _ffn()
    w = [a["w_gate"], a["w_up"], a["w_down"]]
    rest = (None, None, a["dx"], a["h_act"], None, None, a["ws"])
    with pytest.raises(ValueError, match=r"w_down: expected \[64, 128\], got \[128, 64\]"):
        moe.gated_ffn(a["x"], w[0], w[1], w[0], *rest)
    with pytest.raises(ValueError, match=r"w_up: expected \[128, 64\], got \[64, 128\]"):
        moe.gated_ffn(a["x"], w[0], w[2], w[2], *rest)
    with pytest.raises(TypeError, match="w_up"):
        moe.gated_ffn(a["x"], w[0], None, w[2], *rest)
    with pytest.raises(ValueError, match="x: expected"):
        moe.gated_ffn(a["x"][0], *w, *rest)
    with pytest.raises(ValueError, match="x: expected"):
        moe.gated_ffn(None, *w, *rest)


@pytest.mark.parametrize("how", BAD)
@pytest.mark.parametrize("shape", [(2, 24, 40), (24, 40)])
def test_newton_schulz_and_muon_refuse_matrices_of_another_shape(moe, shape, how):
    z = lambda dt=torch.float32: torch.zeros(*shape, dtype=dt)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="out: expected"):
        moe.newton_schulz(z(), _bad(z(), how), ws)
    lr = torch.zeros(1)
    for i, name in enumerate(("w_copy", "momentum", "grad")):
        args = [z(BF), z(), z()]
        args[i] = _bad(args[i], how)
        with pytest.raises(ValueError, match=f"{name}: expected"):
            moe.muon_step(z(), *args, lr, 0.9, 0.0, 1.0, ws)
    with pytest.raises(TypeError, match="momentum"):
        moe.muon_step(z(), z(BF), [1.0], z(), lr, 0.9, 0.0, 1.0, ws)


def test_muon_refuses_a_wrong_gradient_before_any_step(moe, monkeypatch):
    from combine_expert_gemm_gb300 import dense
    stepped = []
    monkeypatch.setattr(dense, "muon_step", lambda *a, **k: stepped.append(a))
    w = [torch.zeros(3, 8, 16), torch.zeros(16, 24)]
    opt = moe.Muon([(t, None) for t in w])
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        opt.step([torch.zeros(3, 8, 16), torch.zeros(24, 16)])
    with pytest.raises(TypeError, match=r"grads\[1\]"):
        opt.step([torch.zeros(3, 8, 16), 0.0])
    assert not stepped
    opt.step([torch.zeros(3, 8, 16), torch.zeros(1, 16, 24)])
    assert len(stepped) == 2
