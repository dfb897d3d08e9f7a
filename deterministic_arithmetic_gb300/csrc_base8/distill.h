/* distill.h -- lora_distill_topk_fwd of include/lora_base8.h with a temperature of 64 bits, for the Python binding: the
 * teacher's probabilities are exponentials of t / T less a log-sum-exp that was made with the caller's T, and where the
 * listed logits have nearly all the mass, T rounded to 24 bits (0.7, say) is what is left of 1 - sum p.
 */
#ifndef DISTILL_H
#define DISTILL_H

#include "../../include/lora_base8.h"

#ifdef __cplusplus
extern "C" {
#endif

lora_status lora_distill_topk_fwd_wide(const void *logits, int type, const void *ids, int id_bytes, const void *teacher,
                                       int teacher_type, const float *teacher_lse, const float *weight, double temperature,
                                       int64_t M, int64_t V, int64_t top, float *loss, float *probs, float *stats,
                                       void *stream);

#ifdef __cplusplus
}
#endif
#endif
