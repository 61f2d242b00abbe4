// C-ABI entry points of the tokens by expert: argument checks and launches.  No
// allocation, no host synchronisation.
#include "../../include/ortho.h"
#include "experts.h"
#include "plan.h"

using namespace ortho;

namespace {

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
ortho_status done(hipError_t e) { return e == hipSuccess ? ORTHO_OK : ORTHO_E_HIP; }

int64_t esz(const ortho_mat& a) { return a.dtype == ORTHO_F32 ? 4 : (a.dtype == ORTHO_BF16 ? 2 : 1); }
const void* data_of(const ortho_mat* a) { return a ? a->data : nullptr; }
int64_t ld_of(const ortho_mat* a) { return a ? a->ld : 0; }
int is_bf(const ortho_mat* a) { return a && a->dtype == ORTHO_BF16; }

ExpertRowsArgs rows_of(const int32_t* slot, const int32_t* offsets, const int32_t* counts, int64_t tokens,
                       int32_t choices, int32_t experts, int64_t rows) {
  return {slot, offsets, counts, static_cast<int>(tokens), choices, experts, rows};
}

}  // namespace

extern "C" {

int64_t ortho_expert_rows(int64_t tokens, int32_t choices, int32_t experts, int32_t align) {
  return expert_rows(tokens, choices, experts, align);
}

size_t ortho_expert_sort_workspace_size(int64_t tokens, int32_t choices, int32_t experts) {
  ExpertSortPlan p;
  return plan_expert_sort(tokens, choices, experts, &p) ? p.total_bytes : 0;
}

ortho_status expert_sort(const void* chosen, int32_t chosen_bytes, int64_t tokens, int32_t choices,
                         int32_t experts, int32_t align, int32_t* slot, int32_t* source,
                         int32_t* offsets, int32_t* counts, void* ws, size_t ws_bytes, void* stream) {
  const ortho_status st = validate_expert_sort(chosen, chosen_bytes, tokens, choices, experts, align, slot, source,
                                               offsets, counts, ws, ws_bytes);
  if (st != ORTHO_OK) return st;
  ExpertSortPlan plan;
  plan_expert_sort(tokens, choices, experts, &plan);
  ExpertSortArgs a{};
  a.chosen = chosen;
  a.wide = chosen_bytes == 8;
  a.pairs = static_cast<int>(plan.pairs);
  a.experts = experts;
  a.align = align;
  a.tiles = plan.tiles;
  a.tile = plan.tile;
  a.slot = slot;
  a.source = source;
  a.offsets = offsets;
  a.counts = counts;
  a.rows = static_cast<int>(expert_rows(tokens, choices, experts, align));
  a.part = static_cast<int32_t*>(ws);
  return done(launch_expert_sort(a, as_stream(stream)));
}

ortho_status expert_gather(ortho_mat X, const ortho_mat* S, const int32_t* slot, int32_t choices,
                           const int32_t* offsets, const int32_t* counts, int32_t experts,
                           ortho_mat Y, const ortho_mat* SY, void* stream) {
  const ortho_status st = validate_expert_gather(X, S, slot, choices, offsets, counts, experts, Y, SY);
  if (st != ORTHO_OK) return st;
  ExpertGatherArgs a{};
  a.r = rows_of(slot, offsets, counts, X.rows, choices, experts, Y.rows);
  a.x = static_cast<const uint8_t*>(X.data);
  a.y = static_cast<uint8_t*>(Y.data);
  a.pitch_x = X.ld * esz(X);
  a.pitch_y = Y.ld * esz(Y);
  a.bytes = X.cols * esz(X);
  if (S) {
    a.s = static_cast<const uint8_t*>(S->data);
    a.sy = static_cast<uint8_t*>(SY->data);
    a.pitch_s = S->ld * esz(*S);
    a.pitch_sy = SY->ld * esz(*SY);
    a.blocks = static_cast<int>(S->cols);
    a.scale_bytes = static_cast<int>(esz(*S));
    while (a.scale_lanes < 8 && 1 << a.scale_lanes < a.blocks) ++a.scale_lanes;
  }
  const Deal d = deal(X.rows, (a.bytes + 15) / 16, 1);
  return done(launch_expert_gather(a, d.lanes, d.across, d.units, as_stream(stream)));
}

ortho_status expert_combine(ortho_mat Y, const int32_t* slot, int32_t choices, const ortho_mat* W,
                            const ortho_mat* Add, ortho_mat Out, void* stream) {
  const ortho_status st = validate_expert_combine(Y, slot, choices, W, Add, Out);
  if (st != ORTHO_OK) return st;
  ExpertCombineArgs a{};
  a.r = rows_of(slot, nullptr, nullptr, Out.rows, choices, 0, Y.rows);
  a.y = Y.data;
  a.ldy = Y.ld;
  a.w = data_of(W);
  a.ldw = ld_of(W);
  a.w_bf = is_bf(W);
  a.add = data_of(Add);
  a.ldadd = ld_of(Add);
  a.add_bf = is_bf(Add);
  a.out = Out.data;
  a.ldout = Out.ld;
  a.n = static_cast<int>(Out.cols);
  const Deal d = deal(Out.rows, Out.cols, 8);
  return done(launch_expert_combine(a, Y.dtype == ORTHO_BF16, d.lanes, d.across, d.units, as_stream(stream)));
}

ortho_status expert_combine_backward(ortho_mat dOut, const int32_t* slot, int32_t choices, const ortho_mat* W,
                                     const int32_t* offsets, const int32_t* counts, int32_t experts, ortho_mat dY,
                                     const ortho_mat* Y, const ortho_mat* dW, void* stream) {
  const ortho_status st =
      validate_expert_combine_backward(dOut, slot, choices, W, offsets, counts, experts, dY, Y, dW);
  if (st != ORTHO_OK) return st;
  ExpertCombineGradArgs a{};
  a.r = rows_of(slot, offsets, counts, dOut.rows, choices, experts, dY.rows);
  a.dout = dOut.data;
  a.lddout = dOut.ld;
  a.w = data_of(W);
  a.ldw = ld_of(W);
  a.w_bf = is_bf(W);
  a.y = data_of(Y);
  a.ldy = ld_of(Y);
  a.dy = dY.data;
  a.lddy = dY.ld;
  a.dw = dW ? static_cast<float*>(dW->data) : nullptr;
  a.lddw = ld_of(dW);
  a.n = static_cast<int>(dOut.cols);
  return done(launch_expert_combine_grad(a, dOut.dtype == ORTHO_BF16, as_stream(stream)));
}

}  // extern "C"
