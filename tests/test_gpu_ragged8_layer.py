"""What the layer over 8-bit pages leaves in them, and over caches long enough for pieces of many key tiles."""
import numpy as np
import pytest
import torch

import oracle as O
from bwd_qwen3_layer_gb300 import layer as L
from bwd_qwen3_layer_gb300 import synth
from _parity import assert_rel
from test_gpu_ragged import D, _dev, _host, _i
from test_gpu_ragged8 import _codes, _f, _step8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1.0, 2.0 ** -6])
def test_layer_scales_and_long_caches(kl, size):
    """Each block's scale after a layer's step: untouched ones keep theirs, a block that the step begins has what its new rows ask for, any
    other the larger of that and what it had. The bf16 layer's pools say what the new rows are (rounded to bf16: off by 2^-8 of
    themselves, so a scale may be that of a size so near). Contexts of up to 20 key tiles, ends inside a tile. size: of what is cached, so
    small that the step's rows make its pages' scales grow, or not."""
    H, Hq, Hkv, I, bs = 256, 16, 2, 512, 16
    reqs = [(1, 2400), (33, 700), (1, 1023), (1, 1024), (3, 1500), (0, 9), (200, 900), (20, 0), (5, 13)]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(23, reqs, Hkv, bs)
    ks, vs = np.nan_to_num(ks, nan=1.0) * size, np.nan_to_num(vs, nan=1.0) * size
    w = synth.layer_weights(22, H, Hq, Hkv, D, I, bf16=True, qk_norm=True)
    cfg = L.make_cfg(1, T, H, Hq, Hkv, D, I, dtype=kl.KL_BF16, qk_norm=True, rope_interleaved=False)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    wd = {k: L.to_device(w[L.SYNTH_NAMES[k]], kl.KL_BF16, "cuda") for k in L.weight_fields(cfg)}
    X = _dev(synth.layer_inputs(22, T, H, bf16=True)["X"])
    pos = np.concatenate([np.arange(c, c + k) for k, c in reqs])
    req = np.repeat(np.arange(len(reqs)), n)
    slots = table[req, pos // bs] * bs + pos % bs
    lens = [_i(table), _i(cu), _i(ctx), _i(pos), _i(slots)]

    def layer(call, size, pools):
        ws = torch.empty(size(cfg, rc), dtype=torch.uint8, device="cuda")
        Y = torch.empty_like(X)
        call(cfg, rc, L.weights_struct(wd), X.data_ptr(), Y.data_ptr(), *[t.data_ptr() for t in pools + lens], ws.data_ptr(), ws.numel())
        assert kl.kl_device_status() == 0
        return Y

    p8 = [_codes(kc), _codes(vc), _f(ks), _f(vs)]
    Y = layer(kl.kl_layer_forward_ragged8, kl.kl_layer_forward_ragged8_ws_bytes, p8)
    k16, v16 = _dev(np.nan_to_num(O.dequantised(kc, ks))), _dev(np.nan_to_num(O.dequantised(vc, vs)))
    Y16 = layer(kl.kl_layer_forward_ragged, kl.kl_layer_forward_ragged_ws_bytes, [k16, v16])
    # (the bound of test_layer_forward)
    assert_rel(_host(Y), _host(Y16), 2.0 ** -4, "Y")
    for s8, x16, old in ((p8[2], k16, ks), (p8[3], v16, vs)):
        got, y = _host(s8), np.abs(_host(x16)).reshape(-1, Hkv, D)
        begun = grown = 0
        for blk in range(nb):
            rows = slots[slots // bs == blk]
            if not len(rows):
                np.testing.assert_array_equal(got[blk], old[blk])
                continue
            a = y[rows].max((0, 2))
            want = [O.scale_for(a * f) for f in (1 - 2.0 ** -7, 1.0, 1 + 2.0 ** -7)]
            if rows.min() % bs:
                assert (got[blk] >= old[blk]).all()
                want = [np.maximum(v, old[blk]) for v in want]
                grown += int((got[blk] > old[blk]).sum())
            else:
                begun += 1
            assert np.any([got[blk] == v for v in want], 0).all(), blk
        assert begun and (grown or size == 1.0)
