"""MI355X-native MoE decode/verify round: a HIP library behind a C ABI, with a thin binding.

    from verify_router_gemv_amd import MoeRound

and the operators such a round calls beside its MoE layers (verify_ops):

    from verify_router_gemv_amd import round_slots, qk_norm_rope, tree_attention, token_logprobs
"""
from .binding import (  # noqa: F401
    LIB_PATH,
    MoeRound,
    MoeRoundError,
    load,
    make_config,
    validate_config,
)
from .verify_ops import (  # noqa: F401
    RoundSlots,
    TokenLogprobs,
    qk_norm_rope,
    round_slots,
    token_logprobs,
    tree_attention,
)
