"""Element types that the Python binding refuses before it calls the library:
what a call would read or write as another type than the tensor's.  (Tensors on
the host: nothing is launched; a call whose types fit is refused for its device.)"""
import pytest
import torch

BF, HALF = torch.bfloat16, torch.float16
B, HQ, HKV, D, NB, W = 3, 8, 2, 64, 10, 4
STORAGE = (torch.int16, torch.uint16)      # two-byte types that hold 16-bit elements when dtype is given


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def zeros(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def args(**over):
    a = dict(q=zeros((B, HQ, D), BF), out=zeros((B, HQ, D), BF), k=zeros((NB, HKV, 16, D), BF),
             v=zeros((NB, HKV, 16, D), BF), k8=zeros((NB, HKV, 16, D), torch.uint8),
             v8=zeros((NB, HKV, 16, D), torch.uint8), ks=zeros(HKV, torch.float32), vs=zeros(HKV, torch.float32),
             tab=zeros((B, W), torch.int32), lens=zeros(B, torch.int32), lists=zeros((B, HKV, 2), torch.int32),
             bounds=zeros((NB, HKV, 2, D), BF), scores=zeros((B, HKV, W), torch.float32), ws=zeros(64, torch.uint8),
             starts=zeros(2, torch.int32), pre=zeros(1, torch.int32), k_new=zeros((B, HKV, D), BF),
             v_new=zeros((B, HKV, D), BF), slots=zeros(B, torch.int64), turns=zeros(D // 2, torch.int64),
             err=zeros(1, torch.int32), dtype=None)
    a.update(over)
    return a


def sparse(pkv, a):
    pkv.pkv_paged_decode_attention_sparse(a["q"], a["k"], a["v"], a["tab"], a["lens"], a["lists"], a["out"], scale=1.0,
                                          workspace=a["ws"], dtype=a["dtype"], err_flag=a["err"], stream=0)


def sparse_fp8(pkv, a, name="pkv_paged_decode_attention_sparse_fp8"):
    getattr(pkv, name)(a["q"], a["k8"], a["v8"], a["ks"], a["vs"], a["tab"], a["lens"], a["lists"], a["out"], scale=1.0,
                       workspace=a["ws"], q_dtype=a["dtype"], err_flag=a["err"], stream=0)


def sparse_e5m2(pkv, a):
    sparse_fp8(pkv, a, "pkv_paged_decode_attention_sparse_e5m2")


def prefix(pkv, a):
    pkv.pkv_paged_decode_attention_prefix(a["q"], a["k"], a["v"], a["tab"], a["lens"], a["starts"], a["pre"], a["out"],
                                          scale=1.0, max_context_len=64, max_prefix_len=16, workspace=a["ws"],
                                          dtype=a["dtype"], err_flag=a["err"], stream=0)


def rope(pkv, a):
    pkv.pkv_rope_append(a["q"], a["k_new"], a["v_new"], a["lens"], a["slots"], a["turns"], a["out"], a["k"], a["v"],
                        dtype=a["dtype"], err_flag=a["err"], stream=0)


def rope_fp8(pkv, a, name="pkv_rope_append_fp8"):
    getattr(pkv, name)(a["q"], a["k_new"], a["v_new"], a["lens"], a["slots"], a["turns"], a["out"], a["k8"], a["v8"],
                       a["ks"], a["vs"], dtype=a["dtype"], err_flag=a["err"], stream=0)


def rope_e5m2(pkv, a):
    rope_fp8(pkv, a, "pkv_rope_append_e5m2")


def rope_keys_alone(pkv, a):
    pkv.pkv_rope_append(None, a["k_new"], a["v_new"], a["lens"], a["slots"], a["turns"], None, a["k"], a["v"],
                        dtype=a["dtype"], err_flag=a["err"], stream=0)


def bounds(pkv, a):
    pkv.pkv_kv_block_bounds(a["k"], a["tab"], a["lens"], a["bounds"], max_new_len=1, dtype=a["dtype"],
                            err_flag=a["err"], stream=0)


def bounds_fp8(pkv, a, name="pkv_kv_block_bounds_fp8"):
    getattr(pkv, name)(a["k8"], a["tab"], a["lens"], a["bounds"], max_new_len=1, dtype=a["dtype"], err_flag=a["err"],
                       stream=0)


def bounds_e5m2(pkv, a):
    bounds_fp8(pkv, a, "pkv_kv_block_bounds_e5m2")


def scores(pkv, a):
    pkv.pkv_block_scores(a["q"], a["bounds"], a["tab"], a["lens"], a["scores"], scale=1.0, max_context_len=64,
                         k_scale=a["ks"], dtype=a["dtype"], err_flag=a["err"], stream=0)


def select(pkv, a):
    pkv.pkv_select_blocks(a["scores"], a["lens"], a["lists"], err_flag=a["err"], stream=0)


# the call's 16-bit tensors, by the name that args() gives them
SIXTEEN = {sparse: "q out k v", sparse_fp8: "q out", sparse_e5m2: "q out", prefix: "q out k v",
           rope: "q out k_new v_new k v", rope_fp8: "q out k_new v_new", rope_e5m2: "q out k_new v_new",
           rope_keys_alone: "k_new v_new k v", bounds: "k bounds", bounds_fp8: "bounds", bounds_e5m2: "bounds",
           scores: "q bounds"}
CALLS = [*SIXTEEN, select]
FP8_OF = {sparse_fp8: torch.float8_e4m3fn, rope_fp8: torch.float8_e4m3fn, bounds_fp8: torch.float8_e4m3fn,
          sparse_e5m2: torch.float8_e5m2, rope_e5m2: torch.float8_e5m2, bounds_e5m2: torch.float8_e5m2}


def refused(pkv, call, a, kinds=(TypeError, ValueError)):
    with pytest.raises(kinds) as e:
        call(pkv, a)
    assert "device" not in str(e.value), e.value


def fits(pkv, call, a):
    with pytest.raises(ValueError, match="device"):
        call(pkv, a)


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_calls_whose_types_fit(pkv, call):
    fits(pkv, call, args())
    fits(pkv, call, args(err=None))
    if call in SIXTEEN:
        names = SIXTEEN[call].split()
        fits(pkv, call, args(**{n: args()[n].half() for n in names}))
        for t in STORAGE:                       # the bits of a 16-bit type, which dtype names
            if call is scores:                  # (q and bounds have one type there)
                continue
            fits(pkv, call, args(dtype=pkv.PKV_F16, **{n: args()[n].view(t) for n in names}))


@pytest.mark.parametrize("call", SIXTEEN, ids=lambda f: f.__name__)
def test_tensors_of_another_16_bit_type(pkv, call):
    names = SIXTEEN[call].split()
    groups = [["k", "v"] if n in "kv" else [n] for n in names]      # (the caches go together)
    for group in groups:
        if len(names) > len(group):
            refused(pkv, call, args(**{n: args()[n].half() for n in group}))
        for t in (torch.uint8, torch.float8_e5m2, torch.int32, torch.float32, torch.float64, *STORAGE):
            refused(pkv, call, args(**{n: torch.zeros(args()[n].shape, dtype=t) for n in group}))


@pytest.mark.parametrize("call", SIXTEEN, ids=lambda f: f.__name__)
def test_a_given_dtype_needs_two_byte_elements(pkv, call):
    names = SIXTEEN[call].split()
    for t in (torch.uint8, torch.float32):
        for n in names:
            refused(pkv, call, args(dtype=pkv.PKV_BF16, **{n: torch.zeros(args()[n].shape, dtype=t)}))
        refused(pkv, call, args(dtype=pkv.PKV_BF16, **{n: torch.zeros(args()[n].shape, dtype=t) for n in names}))


@pytest.mark.parametrize("call", FP8_OF, ids=lambda f: f.__name__)
def test_caches_of_the_other_fp8_format(pkv, call):
    own = FP8_OF[call]
    other = torch.float8_e5m2 if own == torch.float8_e4m3fn else torch.float8_e4m3fn
    shape = args()["k8"].shape
    fits(pkv, call, args(k8=zeros(shape, torch.uint8).view(own), v8=zeros(shape, torch.uint8).view(own)))
    refused(pkv, call, args(k8=zeros(shape, torch.uint8).view(other), v8=zeros(shape, torch.uint8).view(other)),
            TypeError)


@pytest.mark.parametrize("call", [sparse_fp8, sparse_e5m2, rope_fp8, rope_e5m2, scores], ids=lambda f: f.__name__)
def test_scales(pkv, call):
    for name in ("ks",) if call is scores else ("ks", "vs"):
        for bad in (zeros(HKV, HALF), zeros(HKV, torch.float64), zeros(HKV, torch.int32),
                    zeros(2 * HKV, torch.float32)[::2]):
            refused(pkv, call, args(**{name: bad}), TypeError)
        for bad in (zeros(1, torch.float32), zeros(HKV - 1, torch.float32), zeros(HKV + 1, torch.float32)):
            refused(pkv, call, args(**{name: bad}), ValueError)


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_error_flags(pkv, call):
    for bad in (zeros(1, torch.int16), zeros(1, torch.int64), zeros(1, torch.float32), zeros(0, torch.int32)):
        refused(pkv, call, args(err=bad), TypeError)


@pytest.mark.parametrize("call", [sparse, sparse_fp8, prefix], ids=lambda f: f.__name__)
def test_workspaces_that_are_not_one_piece(pkv, call):
    refused(pkv, call, args(ws=zeros(1, torch.uint8).expand(1 << 20)), ValueError)
    refused(pkv, call, args(ws=zeros(128, torch.uint8)[::2]), ValueError)


def test_turns(pkv):
    for bad in (zeros(D // 2, torch.complex64), zeros(D // 2, torch.float64), zeros(D // 2, torch.int32)):
        refused(pkv, rope, args(turns=bad), TypeError)
