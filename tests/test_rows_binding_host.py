"""Host-side checks of the binding (abi.py): a call's rows have to lie as those of
the tensors that its configuration was made from, as the library goes by the
configuration's strides.  No GPU."""
import pytest
import torch

from tests import test_block_ops_host as block
from tests import test_decode_binding_host as byte
from tests.test_decode_binding_host import B, BF16, D, F32, HKV, HQ, I32, T, lib   # noqa: F401
from top_routed_expert_gb300 import abi


def wide(heads, dtype=BF16, more=3):
    """Rows of `heads` heads in a buffer that has more."""
    return torch.zeros(T, heads + more, D, dtype=dtype)[:, :heads]


def calls(call, args, names, dense, apart, lib):   # noqa: F811
    """args(config's rows, call's rows): dense and separate rows, each taken as configured and refused else."""
    good = 0
    for made in (dense, apart):
        for given in (dense, apart):
            if made is given:
                call(**args(made, given))
                good += 1
            else:
                with pytest.raises(ValueError, match=names[0]):
                    call(**args(made, given))
    assert lib.calls == good


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["k_out", "v_out"])
def test_read(lib, dtype, name):   # noqa: F811
    def args(made, given):
        a = block.read_args(dtype=dtype)
        rows = dict(k_out=a["k_out"], v_out=a["v_out"])
        return dict(a, cfg=abi.make_blockkv_read_config(*dict(rows, **{name: made}).values(), B), **{name: given})
    dense, apart = torch.zeros(T, HKV, D, dtype=dtype), wide(HKV, dtype)
    calls(abi.moe_blockkv_read, args, [name], dense, apart, lib)
    done = lib.calls
    # the whole buffer has the slice's rows; the same strides with fewer rows, or longer ones of another shape, have not
    abi.moe_blockkv_read(**args(apart, apart._base))
    abi.moe_blockkv_read(**args(dense, dense.flatten(1)))
    abi.moe_blockkv_read(**args(dense, torch.zeros(T + 4, HKV, D, dtype=dtype)))
    for made, given in ((apart, apart[:T - 1]), (apart, apart._base[:T - 1]), (dense, apart[:, :, :D // 2]), (dense, dense[:T - 1]),
                        (apart, torch.zeros(T, HKV + 3, D, dtype=dtype).transpose(0, 1))):
        with pytest.raises(ValueError, match=name):
            abi.moe_blockkv_read(**args(made, given))
    assert lib.calls == done + 3


def test_read_of_one_row(lib):   # noqa: F811
    """A single row may carry any distance to a next one."""
    a = block.read_args()
    for made in (a["k_out"][:1], wide(HKV)[:1]):
        cfg = abi.make_blockkv_read_config(made, made, B)
        for given in (a["k_out"][:1], wide(HKV)[:1], a["k_out"][0]):
            abi.moe_blockkv_read(**dict(a, cfg=cfg, k_out=given, v_out=given))
    assert lib.calls == 6


APPENDS = [(abi.moe_kv_append, byte.append_args), (abi.moe_blockkv_append, block.append_args)]
ATTENTIONS = [(abi.moe_paged_attention, byte.attend_args), (abi.moe_blockkv_attention, block.attend_args)]


@pytest.mark.parametrize("call,args", APPENDS)
@pytest.mark.parametrize("name", ["q", "k", "v", "q_out"])
def test_append(lib, call, args, name):   # noqa: F811
    heads = HQ if name in ("q", "q_out") else HKV

    def given(made, rows):
        a = args()
        own = dict({n: a[n] for n in ("q", "k", "v", "q_out")}, **{name: made})
        return dict(a, cfg=abi.make_kv_append_config(*own.values(), B, rot_dim=D, n_pos=50), **{name: rows})
    dense, apart = torch.zeros(T, heads, D, dtype=BF16), wide(heads)
    calls(call, given, [name], dense, apart, lib)
    done = lib.calls
    call(**given(apart, apart._base))
    call(**given(dense, dense.flatten(1)))
    for made, bad in ((apart, apart._base[:T - 1]), (dense, dense.float()), (dense, dense.half()), (apart, wide(heads, F32))):
        with pytest.raises(ValueError, match=name):
            call(**given(made, bad))
    assert lib.calls == done + 2


@pytest.mark.parametrize("call,args", APPENDS)
def test_slices_of_one_projection(lib, call, args):   # noqa: F811
    a = args()
    x = torch.zeros(T, (HQ + 2 * HKV) * D, dtype=BF16)
    q, k, v = (y.unflatten(1, (-1, D)) for y in x.split([HQ * D, HKV * D, HKV * D], dim=1))
    cfg = abi.make_kv_append_config(q, k, v, a["q_out"], B, rot_dim=D, n_pos=50)
    call(**dict(a, cfg=cfg, q=q, k=k, v=v))
    cfg.T = T - 2
    call(**dict(a, cfg=cfg, q=q[:T - 2], k=k[:T - 1], v=v))
    with pytest.raises(ValueError, match="q_out"):
        call(**dict(a, cfg=cfg, q=q[:T - 3], k=k, v=v))
    assert lib.calls == 2


@pytest.mark.parametrize("call,args", ATTENTIONS)
@pytest.mark.parametrize("name", ["q", "out"])
def test_attention(lib, call, args, name):   # noqa: F811
    def given(made, rows):
        a = args()
        own = dict({n: a[n] for n in ("q", "out")}, **{name: made})
        return dict(a, cfg=abi.make_paged_attention_config(*own.values(), B), **{name: rows})
    dense, apart = torch.zeros(T, HQ, D, dtype=BF16), wide(HQ)
    calls(call, given, [name], dense, apart, lib)
    done = lib.calls
    call(**given(apart, apart._base))
    call(**given(dense, dense.flatten(1)))
    for made, bad in ((apart, apart._base[:T - 1]), (dense, dense.float()), (dense, dense.half()), (apart, wide(HQ, F32))):
        with pytest.raises(ValueError, match=name):
            call(**given(made, bad))
    assert lib.calls == done + 2


@pytest.mark.parametrize("name", ["x", "residual", "out", "sum"])
def test_norm(lib, name):   # noqa: F811
    dtype = BF16 if name in ("x", "out") else F32

    def given(made, rows):
        a = block.norm_args()
        own = dict({n: a[n] for n in ("x", "residual", "out", "out8", "sum")}, **{name: made})
        return dict(a, cfg=abi.make_add_rms_norm_config(*own.values(), group=128), **{name: rows})
    dense, apart = torch.zeros(T, 512, dtype=dtype), torch.zeros(T, 1024, dtype=dtype)[:, :512]
    calls(abi.moe_add_rms_norm, given, [name], dense, apart, lib)
    done = lib.calls
    abi.moe_add_rms_norm(**given(apart, apart._base))
    abi.moe_add_rms_norm(**given(dense, dense.flatten()))
    for bad in (apart._base[:T - 1], apart._base[:T - 2], torch.zeros(2 * T, 1024, dtype=dtype)[:, :504]):
        with pytest.raises(ValueError, match=name):
            abi.moe_add_rms_norm(**given(apart, bad))
    assert lib.calls == done + 2


@pytest.mark.parametrize("call,args,names", [
    (abi.moe_route_scores, byte.route_args, ("bias", "topk_ids", "topk_w")),
    *((c, a, ("gamma_q", "gamma_k", "cos_sin", "positions", "cu", "kv_len")) for c, a in APPENDS),
    *((c, a, ("cu", "kv_len", "lse", "ws")) for c, a in ATTENTIONS),
    (abi.moe_blockkv_read, block.read_args, ("cu", "kv_len")),
])
def test_arrays_with_gaps(lib, call, args, names):   # noqa: F811
    for name in names:
        t = args()[name]
        gaps = torch.zeros(*t.shape, 2, dtype=t.dtype)[..., 0]
        with pytest.raises(ValueError, match=name):
            call(**args(**{name: gaps}))
        call(**args(**{name: gaps.contiguous()}))
    assert lib.calls == len(names)
