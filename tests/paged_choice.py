"""Which attention kernel a call of the many-request operators takes, by its bounds: the rule of
csrc/paged_api.cu, written again so that a test can say which kernel it is about."""
SMS, FEW_ROWS, TILE_ROWS = 148, 32, 256


def tiles(p, paged):
    """True: the tile kernel, where keys and values have strides that it takes."""
    group = p.n_heads // p.n_kv_heads
    cols = p.max_blocks * p.page_size if paged else min(p.max_new, p.max_tokens)
    if min(p.max_new, p.max_tokens) * group <= FEW_ROWS or cols > 1 << 24:
        return False
    rows, requests = p.max_tokens * p.n_heads, min(p.batch, p.max_tokens)
    starts = requests * p.n_kv_heads / 2
    few, some = rows / FEW_ROWS + starts, rows / TILE_ROWS + starts
    stages, units = (cols + 63) // 64, (cols + 127) // 128
    stage, unit = (1.4, 1.9) if p.head_dim == 128 else (0.6, 1.6)
    if not paged:
        few_us = max(3.0 + stage * stages, few / (2 * SMS) * (7.5 + stage / 2 * stages))
        return max(7.0 + unit * units, some / SMS * (7.0 + unit / 2 * units)) < few_us
    hbm = requests * cols * p.n_kv_heads * p.head_dim * 4 / 6.5e6
    if cols <= 512:
        few_us = max(3.0 + stage * stages, few / (2 * SMS) * (7.5 + stage * stages))
    else:
        few_us = 9.0 + max(1.2 * stage * max(4.0, few * (stages + 6) / (2 * SMS)), 1.15 * hbm)
    return 18.0 + max(1.05 * unit * max(4.0, some * (units + 2) / SMS), 1.35 * hbm) < few_us


def scratch(p):
    """Bytes that flashloop_paged_attn asks for: the two kernels' differ."""
    def at(*sizes):
        total = 0
        for n in sizes:
            total += -(-n // 256) * 256
        return total
    if tiles(p, True):
        return at(SMS * 32, 2 * SMS * TILE_ROWS * 8, 2 * SMS * TILE_ROWS * p.head_dim * 4)
    if p.max_blocks * p.page_size > 512:
        return at(2 * SMS * 32, 4 * SMS * FEW_ROWS * 8, 4 * SMS * FEW_ROWS * p.head_dim * 4)
    return 16
